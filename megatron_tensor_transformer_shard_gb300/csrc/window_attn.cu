// Head-local causal attention over a sliding window with sink tokens, for packed sequences, on
// tcgen05: forward and backward ("02 — Tensor Parallelism", "The attention pairing": each shard
// runs its own heads, no communication).  Query q of a sequence that begins at st sees the keys
// j with st <= j <= q and (q - j < W or j - st < S):
//   s_j = scale q . k_j,  p = softmax(s),  o = sum p_j v_j,  lse = log sum e^s_j,
//   dV = P^T dO,  dP = dO V^T,  dS = P (dP - D),  D = rowsum(dO O),  dQ = scale dS K,  dK = scale dS^T Q.
//
// Bound by the tensor cores (4 x 128 flops a visible pair forward, 10 x 128 backward, where the two
// kernels run 14 x 128 as each forms the scores and dP again), so the design is that of the full
// causal kernels (attention.cu: fp16
// operands, S, P, dS and the accumulators in TMEM, K / V streamed by TMA) over a shorter list of
// key blocks: the blocks that hold sinks, then the blocks that the window of the tile's first
// row reaches, up to the diagonal.  Only a tile's first row can belong to a sequence that began
// before the tile; sequences that begin inside it have their keys in the diagonal block.  So one
// pair of block ranges, taken from the first row, covers a tile whatever the packing, and rows
// mask the rest by their own intervals, as a bit mask per 32 scores (one test per score; four
// comparisons per score made the masked blocks, a third of all at W = 1024, the slow ones).
//
// Forward tiles work in pairs, so that one's softmax runs while the other's MMAs do.  With
// grouped-query heads (an even group) the pair is two query heads of one KV head over the same
// queries: both read the same key blocks, none is loaded for one tile only.  Otherwise it is
// two neighbouring query tiles of one head.
//
// Sinks in the backward: the key block with a sequence's sinks is seen by all of its queries,
// N / 64 blocks of them against (W + 128) / 64 for the others; one CTA would run alone long
// after the rest.  The queries beyond the window's reach of a sink block are cut into chunks of
// at most max(W, 128) rows: then, of the sequences in a chunk, only the one that its first row
// belongs to can have such queries in it.  One work per (KV head, chunk, sink block) leaves fp32
// dK, dV of the sink rows in the workspace, as the sink block's own work does, and a last small
// kernel adds them in chunk order: no atomics, the same bits every time.  The chunk works come
// first in the launch of the key blocks (as a launch of their own, 100 long works on 152 SMs,
// they took 153 us of 2373 at N 16384, 64 / 8 heads, W 1024).
//
// The MMA thread is an elected one (ptx::elect_one): behind `lane == 0` an MMA took it some 65 cycles,
// as long as the tensor cores take to run it, and its pauses were theirs (N 16384, 64 / 8 heads, W 1024,
// seven sequences, forward and backward: 2296 us, elected 1857).
//
// Measured, 64 / 8 heads, N 16384: forward W 1024, 16 sinks 466 us (1163 TFLOP/s of visible pairs; the
// 128-key blocks at the two edges and the sinks' make it 10 blocks where 8 would hold the window), full
// causal 2560 us (1718); dQ 703 us, dK / dV 842 us at W 1024 (SM throughput 79 and 85 %).
//
// P and dS are rounded to fp16 (2^-11, relative) because the MMA takes 16-bit operands; scores, row
// maxima and sums, lse, D and every accumulator stay fp32.  Near zero fp16 has 2^-25 absolute.  Against
// the forward's row sum of at least 1 that is nothing; but a row of P under a wide window, and dS with
// dO's magnitude in it, may lie there altogether.  So the backward holds P 2^13 and dS 2^e, and takes the
// powers of two out with the fp32 results: they shift exponents, and change no other bit.  |dO . v| is
// at most B = max|dO| max sum|v|, |D| as much (and 2^-8 for O's rounding), so e = 13 - floor(log2 B)
// keeps |dS| 2^e below 33,000, all bits of what is above 2^-27 B, and steps of 2^-37 B below, whatever the
// magnitudes of dO and V.  dQ has an e for every 32 query rows, with the v's of the key blocks that their tile
// sees; dK sums over queries, so it has one for each KV head, from the largest B of all rows.
// Before dQ, window_prep_kernel takes the largest sum|v| of each key block; it, and then the largest
// B of a KV head, wait in places of the outputs that are free at the time: value_bound(), row_bound().
// Measured, backward at N 16384, 64 / 8 heads, W 1024, seven sequences, and at N 2048, 96 / 96 heads, W 512:
// 1384 and 222 us with dS as it was, 1407 and 233 so.
#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_runtime.h>

#include <cfloat>
#include <climits>
#include <cmath>
#include <type_traits>

#include "attn_tiles.cuh"
#include "devmath.cuh"
#include "internal.h"
#include "ptx.cuh"

namespace tp {
namespace {

constexpr int FWD_THREADS = 320;  // TMA warp, MMA warp, two softmax warpgroups
constexpr int KV_SLOTS = 5;       // K and V tiles share one ring
constexpr int QUEUE_SMEM = 192;   // WorkQueue
constexpr int FWD_SMEM = 1024 + (2 + KV_SLOTS) * TILE + 256 + QUEUE_SMEM;
constexpr float kLazyRescale = 8.0f;
// Reference maximum of a row that has seen no key yet.  Finite: with -inf, a block in which the
// row sees nothing would rescale by 2^(-inf + inf).
constexpr float kNoMax = -3.0e38f;

enum : int { ERR_WIN_PRODUCER = 0x151, ERR_WIN_MMA = 0x152, ERR_WIN_SOFTMAX = 0x153, ERR_WIN_DRAIN = 0x154 };
constexpr int kErrSeqlens = 0x202;  // cu_seqlens not 0 <= .. non-decreasing .. <= N

struct WinArgs {
  int N, H, hpr, Gs, kv_t, Hkv;
  int W, S;              // window and sinks, at most N
  int by_head;           // forward: a pair of tiles is two heads of one group
  int nqb;               // 128-row blocks
  int64_t dt;            // width of one shard's Q block (and of its O)
  int64_t row_w, kcol0, vcol0;
  float scale, scale_log2;
  const int2* span;      // [N] (begin, end) of each row's sequence, end <= row: none; NULL: one sequence
  const int* total;      // rows that belong to a sequence; NULL: N
  const uint16_t* QKV;   // [t][N][row_w]
  uint16_t* O;           // [t][N][dt]
  float* lse;            // [t][hpr][N]
  int wide;              // O (backward: dQKV) is 32-byte aligned
  int zero_pad;          // forward: write zeros to the rows behind the last sequence
  // backward
  const uint16_t* dO;    // as O
  float* Dvec;           // [t][hpr][N], written by the dQ kernel
  uint16_t* dQKV;
  int dqkv_f16;
  float* far;            // [Hkv][2 nch][S][2][128] dV, dK of the sinks: far_row()
  int C, nch, nsb, nfar; // rows of a chunk, chunks, sink blocks a sequence can have, far works; nch = 0: no far queries
  int* err;
  uint64_t timeout_ns;
};

// Plain loads, as for all that an earlier kernel writes: this one may have started before it was done, so its data is
// not read-only for the whole kernel, as a non-coherent load would need.
__device__ __forceinline__ int total_rows(const WinArgs& p) { return p.total ? *p.total : p.N; }
__device__ __forceinline__ int2 span_of(const WinArgs& p, int row) {
  if (row >= p.N) return make_int2(row, row);
  return p.span ? p.span[row] : make_int2(0, p.N);
}

// Key blocks (of 2^LOG keys) that the 128 queries from q0 see: [a0, a1) hold sinks behind the
// window, [b0, b1) the window, a1 <= b0.  Empty when row q0 belongs to no sequence.
struct KeyBlocks {
  int a0, a1, b0, b1;
  __device__ bool has(int x) const { return (x >= a0 && x < a1) || (x >= b0 && x < b1); }
  // the first block >= x, INT_MAX when there is none
  __device__ int from(int x) const {
    if (x < a1) return max(x, a0);
    if (x < b1) return max(x, b0);
    return INT_MAX;
  }
};
template <int LOG>
__device__ __forceinline__ KeyBlocks key_blocks(const WinArgs& p, int q0, int total) {
  KeyBlocks l{0, 0, 0, 0};
  const int2 sp = span_of(p, q0);
  if (sp.y <= q0) return l;
  const int last = min(q0 + 127, total - 1);
  l.b0 = max(sp.x, q0 - p.W + 1) >> LOG;
  l.b1 = (last >> LOG) + 1;
  if (p.S > 0) {
    l.a0 = sp.x >> LOG;
    l.a1 = min((min(sp.x + p.S - 1, last) >> LOG) + 1, l.b0);
    if (l.a1 <= l.a0) l.a0 = l.a1 = 0;
  }
  return l;
}

// Bits lo..hi (inclusive, clipped) of a 32-bit word.
__device__ __forceinline__ uint32_t span_bits(int lo, int hi) {
  lo = max(lo, 0);
  hi = min(hi, 31);
  return hi < lo ? 0u : (0xffffffffu >> (31 - hi)) & (0xffffffffu << lo);
}

// One query row once more on the CUDA cores, by a whole warp, over its visible keys only.  The
// tensor cores multiply the P = 0 of a hidden key with that key's values; a non-finite value
// there (another sequence's, or a later token's) makes the row NaN.  Rows that come out
// non-finite are therefore formed again here: they stay NaN only if something they see is.
__device__ __noinline__ void slow_row(const WinArgs& p, int shard, int qcol, int kcol, int vcol, int q, int st,
                                      uint16_t* orow, float* lse) {
  const int lane = threadIdx.x & 31;
  const uint16_t* rows = p.QKV + static_cast<int64_t>(shard) * p.N * p.row_w + 4 * lane;
  float qv[4], m = -INFINITY, l = 0.0f, o[4] = {0.f, 0.f, 0.f, 0.f};
  const uint2 qw = *reinterpret_cast<const uint2*>(rows + static_cast<int64_t>(q) * p.row_w + qcol);
  unpack_f16x2(qw.x, qv[0], qv[1]);
  unpack_f16x2(qw.y, qv[2], qv[3]);
  const int s_end = min(st + p.S, q + 1);                 // sinks [st, s_end)
  const int w0 = max(max(st, q - p.W + 1), s_end);        // then the window's keys behind them
  for (int j = (s_end > st ? st : w0); j <= q; j = (j + 1 == s_end ? w0 : j + 1)) {
    const uint16_t* row = rows + static_cast<int64_t>(j) * p.row_w;
    const uint2 kw = *reinterpret_cast<const uint2*>(row + kcol), vw = *reinterpret_cast<const uint2*>(row + vcol);
    float k[4], v[4];
    unpack_f16x2(kw.x, k[0], k[1]);
    unpack_f16x2(kw.y, k[2], k[3]);
    unpack_f16x2(vw.x, v[0], v[1]);
    unpack_f16x2(vw.y, v[2], v[3]);
    float s = fmaf(qv[0], k[0], fmaf(qv[1], k[1], fmaf(qv[2], k[2], qv[3] * k[3])));
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
    s *= p.scale_log2;
    const float mn = fmaxf(m, s);
    const float al = exp2f(m - mn), e = exp2f(s - mn);  // NaN when s is, or when every score so far is -inf
    l = fmaf(l, al, e);
#pragma unroll
    for (int c = 0; c < 4; ++c) o[c] = fmaf(o[c], al, e * v[c]);
    m = mn;
    if (l != l) break;  // the row is NaN
  }
  const float inv = 1.0f / l;
  uint2 w;
  w.x = pack_bf16x2(o[0] * inv, o[1] * inv);
  w.y = pack_bf16x2(o[2] * inv, o[3] * inv);
  if (l != l) w = make_uint2(0x7fc07fc0u, 0x7fc07fc0u);
  *reinterpret_cast<uint2*>(orow + 4 * lane) = w;
  if (lane == 0) *lse = (m + log2f(l)) * kLn2;
}

// Offset of k-step kk (16 columns) of a K-major tile in two 64-column panels.
__device__ __forceinline__ constexpr int kstep(int kk, int panel) { return (kk >> 2) * panel + (kk & 3) * 32; }

// Running maxima over 32 scores.
__device__ __forceinline__ void max32(const uint32_t (&r)[32], float (&mx4)[4]) {
#pragma unroll
  for (int e = 0; e < 32; e += 8) {
    mx4[0] = max3f(mx4[0], __uint_as_float(r[e]), __uint_as_float(r[e + 1]));
    mx4[1] = max3f(mx4[1], __uint_as_float(r[e + 2]), __uint_as_float(r[e + 3]));
    mx4[2] = max3f(mx4[2], __uint_as_float(r[e + 4]), __uint_as_float(r[e + 5]));
    mx4[3] = max3f(mx4[3], __uint_as_float(r[e + 6]), __uint_as_float(r[e + 7]));
  }
}
// P = 2^(s scale - m) of 32 scores as fp16 pairs, added to the running row sums: two scores an instruction.
__device__ __forceinline__ void exp32(const uint32_t (&r)[32], float sl2, float neg_m, uint64_t (&rs2)[2],
                                      uint32_t (&wd)[16]) {
  const uint64_t sl2x2 = f2_pack(sl2, sl2), negm2 = f2_pack(neg_m, neg_m);
#pragma unroll
  for (int e = 0; e < 16; ++e) {
    float x0, x1;
    f2_unpack(f2_fma(f2_pack(__uint_as_float(r[2 * e]), __uint_as_float(r[2 * e + 1])), sl2x2, negm2), x0, x1);
    const float p0 = ptx::exp2_approx(x0), p1 = ptx::exp2_approx(x1);
    rs2[e & 1] = f2_add(rs2[e & 1], f2_pack(p0, p1));
    wd[e] = pack_f16x2(p0, p1);
  }
}
// Hidden scores become -inf.
__device__ __forceinline__ void mask32(uint32_t (&r)[32], uint32_t bits) {
#pragma unroll
  for (int e = 0; e < 32; ++e) r[e] = (bits >> e) & 1u ? r[e] : 0xff800000u;
}
// Maximum and P under a scale that is not positive (or so small that it may count as 0): scores and scale
// are negated, and hidden scores are left out by selection, as -inf * 0 would be NaN.
__device__ __forceinline__ void max32_neg(const uint32_t (&r)[32], uint32_t bits, float (&mx4)[4]) {
#pragma unroll
  for (int e = 0; e < 32; ++e) mx4[e & 3] = fmaxf(mx4[e & 3], (bits >> e) & 1u ? -__uint_as_float(r[e]) : -INFINITY);
}
__device__ __forceinline__ void exp32_neg(const uint32_t (&r)[32], uint32_t bits, float sl2, float neg_m,
                                          uint64_t (&rs2)[2], uint32_t (&wd)[16]) {
#pragma unroll
  for (int e = 0; e < 32; e += 2) {
    float p0 = ptx::exp2_approx(fmaf(-__uint_as_float(r[e]), sl2, neg_m));
    float p1 = ptx::exp2_approx(fmaf(-__uint_as_float(r[e + 1]), sl2, neg_m));
    p0 = (bits >> e) & 1u ? p0 : 0.0f;
    p1 = (bits >> (e + 1)) & 1u ? p1 : 0.0f;
    rs2[(e >> 1) & 1] = f2_add(rs2[(e >> 1) & 1], f2_pack(p0, p1));
    wd[e >> 1] = pack_f16x2(p0, p1);
  }
}
// 32 bytes to a 32-byte aligned address in one store.
__device__ __forceinline__ void st_global_32b(uint16_t* dst, const uint32_t* v) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(dst), "r"(v[0]), "r"(v[1]), "r"(v[2]),
               "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
               : "memory");
}

// A wait of all lanes of a warp: they go on, or give up, together, as votes and shuffles follow.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, volatile int* abort_flag, int* err, int code,
                                          uint64_t limit_ns) {
  return __all_sync(0xffffffffu, ptx::mbar_wait(bar, parity, abort_flag, err, code, limit_ns));
}

// The works of a persistent CTA: its own block index, then those of CTAs that had not started, taken over
// one at a time, so that works of different length (sequence ends, the last rows) spread evenly: dealing
// them out by stride left the longest CTA 9 to 20 % above the mean.  The producer asks for the next one
// once it has issued the loads of the one before, a few tiles ahead of the MMAs (asking when a work began
// gave a CTA its second long one while others had none; asking two steps earlier made dK / dV 3 % slower, and
// the forward no faster).  It alone finds the work's blocks (divisions, dependent loads of sequence bounds)
// and passes them on in two slots in turn, so no other role has that between its last block and its first
// (N 16384, 64 / 8 heads, W 1024: forward 471 us, 479 when each role found them).
template <class Work, int CONSUMERS>  // the MMA thread, a lane of each warp that reads TMEM
struct WorkQueue {
  static constexpr int SMEM = QUEUE_SMEM;
  uint8_t* answer;   // 16 bytes, 16-byte aligned
  uint64_t* asked;   // the answer is there
  uint64_t* full;    // [2]
  uint64_t* empty;   // [2]
  Work* slot;        // [2]
  uint32_t i, asks;  // works posted or read, asked for
  bool pending;
  __device__ WorkQueue(uint8_t* smem)
      : answer(smem), asked(reinterpret_cast<uint64_t*>(smem + 16)), full(reinterpret_cast<uint64_t*>(smem + 24)),
        empty(reinterpret_cast<uint64_t*>(smem + 40)), slot(reinterpret_cast<Work*>(smem + 56)), i(0), asks(0),
        pending(false) {
    static_assert(56 + 2 * sizeof(Work) <= SMEM && alignof(Work) <= 8, "room for two works");
  }
  __device__ void init() {
    ptx::mbar_init(asked, 1);
    for (int s = 0; s < 2; ++s) {
      ptx::mbar_init(&full[s], 1);
      ptx::mbar_init(&empty[s], CONSUMERS);
    }
  }
  // Producer: ask for another work, unless that was done.
  __device__ void ask() {
    if (pending) return;
    ptx::fence_proxy_async_smem();  // the old answer was read before the new one is written
    ptx::mbar_arrive_expect_tx(asked, 16);
    ptx::clc_try_cancel(answer, asked);
    pending = true;
  }
  // .. and its index, -1 when there is none (or the wait was given up).
  __device__ int next(volatile int* abort_flag, int* err, int code, uint64_t limit_ns) {
    ask();
    if (!ptx::mbar_wait(asked, asks & 1, abort_flag, err, code, limit_ns)) return -1;
    pending = false;
    ++asks;
    return ptx::clc_answer(answer);
  }
  // Producer, before the CTA exits: an answer on its way lands first.
  __device__ void drain(int* err, int code, uint64_t limit_ns) {
    volatile int never = 0;
    if (pending) ptx::mbar_wait(asked, asks & 1, &never, err, code, limit_ns);
  }
  // Producer: pass a work on (shard -1: there are no more).
  __device__ bool post(const Work& k, volatile int* abort_flag, int* err, int code, uint64_t limit_ns) {
    if (!ptx::mbar_wait(&empty[i & 1], ((i >> 1) & 1) ^ 1u, abort_flag, err, code, limit_ns)) return false;
    slot[i & 1] = k;
    ptx::mbar_arrive(&full[i & 1]);
    ++i;
    return true;
  }
  __device__ bool post_end(volatile int* abort_flag, int* err, int code, uint64_t limit_ns) {
    Work k;
    k.shard = -1;
    return post(k, abort_flag, err, code, limit_ns);
  }
  // The next work, for one thread or for all lanes of a warp.  False: no more, or given up.
  template <bool WARP>
  __device__ bool read(Work& k, volatile int* abort_flag, int* err, int code, uint64_t limit_ns) {
    if (!(WARP ? warp_wait(&full[i & 1], (i >> 1) & 1, abort_flag, err, code, limit_ns)
               : ptx::mbar_wait(&full[i & 1], (i >> 1) & 1, abort_flag, err, code, limit_ns)))
      return false;
    k = slot[i & 1];
    if (WARP) __syncwarp();
    if (!WARP || (threadIdx.x & 31) == 0) ptx::mbar_arrive(&empty[i & 1]);
    ++i;
    return k.shard >= 0;
  }
};

// Where the sequence of `rows` rows from r0 begins, -1 when it is not one for all of them.
__device__ __forceinline__ int common_begin(const WinArgs& p, int r0, int rows, int total) {
  const int last = min(r0 + rows, total) - 1, begin = span_of(p, r0).x;
  return last >= r0 && span_of(p, last).x == begin ? begin : -1;
}

// One pair of query tiles: query blocks qb0 and qb0 + qstep, heads jj0 and jj0 + hstep of a shard.
// Late query blocks (the ones with a full window) come first.
struct FwdWork {
  int shard, jj0, qb0, kcol, vcol;
  KeyBlocks l0, l1;
  int st0, st1;  // where the sequence of the tile's rows begins, -1: not one for all rows
  FwdWork() = default;
  __device__ FwdWork(const WinArgs& p, int w, int npair, int total) {
    const int first = (w % npair) * (p.by_head ? 2 : 1);
    shard = first / p.hpr;
    jj0 = first - shard * p.hpr;
    const int nsb = p.by_head ? p.nqb : (p.nqb + 1) / 2;
    const int sb = nsb - 1 - w / npair;
    qb0 = p.by_head ? sb : 2 * sb;
    kcol = static_cast<int>(p.kcol0) + (jj0 / p.Gs) * HD;  // the KV head of both tiles
    vcol = static_cast<int>(p.vcol0) + (jj0 / p.Gs) * HD;
    l0 = key_blocks<7>(p, qb0 * BQ, total);
    l1 = p.by_head ? l0 : key_blocks<7>(p, (qb0 + 1) * BQ, total);
    st0 = common_begin(p, qb0 * BQ, BQ, total);
    st1 = p.by_head ? st0 : common_begin(p, (qb0 + 1) * BQ, BQ, total);
  }
  __device__ int next(int x) const { return min(l0.from(x), l1.from(x)); }
};

// Persistent: one CTA an SM walks the pairs that its queue gives.  A pair has only about W / 128
// key blocks, and a CTA of its own spent 9 us on its first loads, its last softmax and its output (246 of
// 624 us at N 16384, 64 heads, W 1024, before any of the steps below); here the next pair's Q, K and S run
// meanwhile.  (Output warps of their own leave 128 registers a thread: 441 us where this takes 400, packed
// N 15937, and 2888 for 2535 full causal.)  Counters that
// give barrier phases run on over the pairs: key tiles of the ring, blocks of each query tile, pairs.
template <bool NEG>
__global__ void __launch_bounds__(FWD_THREADS, 1)
    window_fwd_kernel(const __grid_constant__ CUtensorMap tm_qkv, const __grid_constant__ WinArgs p) {
  extern __shared__ uint8_t dsmem[];
  const uint32_t pad = (1024u - (ptx::smem_addr(dsmem) & 1023u)) & 1023u;
  uint8_t* base = dsmem + pad;
  uint8_t* sQ = base;              // two query tiles
  uint8_t* sKV = base + 2 * TILE;  // ring of KV_SLOTS tiles: K_0, V_0, K_1, V_1, ...
  uint64_t* bars = reinterpret_cast<uint64_t*>(base + (2 + KV_SLOTS) * TILE);
  uint64_t* q_full = bars + 0;
  uint64_t* q_empty = bars + 1;                 // the pair's last S read Q
  uint64_t* kv_full = bars + 2;                 // [KV_SLOTS]
  uint64_t* kv_empty = bars + 2 + KV_SLOTS;     // [KV_SLOTS]
  uint64_t* s_full = bars + 2 + 2 * KV_SLOTS;   // [2] S_b ready in TMEM
  uint64_t* p_full = bars + 4 + 2 * KV_SLOTS;   // [2] P_b written over S_b,
  uint64_t* o_full = bars + 6 + 2 * KV_SLOTS;   // [2] last P_b V of the pair done
  uint64_t* o_empty = bars + 8 + 2 * KV_SLOTS;  // [2] O_b read
  uint64_t* p_half = bars + 10 + 2 * KV_SLOTS;  // [2] .. its keys 64-127
  uint64_t* mma_done = bars + 12 + 2 * KV_SLOTS;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 13 + 2 * KV_SLOTS);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  WorkQueue<FwdWork, 9> queue(reinterpret_cast<uint8_t*>(bars) + 256);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    ptx::mbar_init(q_full, 1);
    ptx::mbar_init(q_empty, 1);
    for (int s = 0; s < KV_SLOTS; ++s) {
      ptx::mbar_init(&kv_full[s], 1);
      ptx::mbar_init(&kv_empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      ptx::mbar_init(&s_full[b], 1);
      ptx::mbar_init(&p_full[b], 4);
      ptx::mbar_init(&p_half[b], 4);
      ptx::mbar_init(&o_full[b], 1);
      ptx::mbar_init(&o_empty[b], 128);
    }
    ptx::mbar_init(mma_done, 1);
    queue.init();
    *abort_flag = 0;
    ptx::fence_mbar_init();
  }
  if (warp == 1) {
    ptx::tmem_alloc(tmem_slot, 512);
    ptx::tmem_relinquish();
  }
  ptx::tc_fence_before();
  __syncwarp();  // lane-0 roles rejoin their warp: bar.sync needs converged warps
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  // Programmatic dependent launch: nothing that an earlier kernel writes is read above.
  ptx::griddep_wait();
  ptx::griddep_launch_dependents();
  const int total = total_rows(p);
  const int qstep = p.by_head ? 0 : 1, hstep = p.by_head ? 1 : 0;
  // Every role may come to wait for softmax warps that are in slow_row (about 60 cycles a visible key and
  // row): a limit that allows for some ten million keys.
  const uint64_t patient_ns = 16 * p.timeout_ns;

  // TMEM columns: S_0 | S_1 | O_0 | O_1, 128 each.  P_b (fp16 pairs) overwrites the last 64 columns of S_b.
  if (warp == 0) {
    if (lane == 0) {
      ptx::tma_prefetch_desc(&tm_qkv);
      uint32_t issued = 0, pairs = 0;
      bool ok = true;
      const int npair = p.by_head ? p.H / 2 : p.H;
      for (int w = blockIdx.x; ok && w >= 0; w = queue.next(abort_flag, p.err, ERR_WIN_PRODUCER, patient_ns)) {
        const FwdWork k(p, w, npair, total);
        if (!queue.post(k, abort_flag, p.err, ERR_WIN_PRODUCER, patient_ns)) {
          ok = false;
          break;
        }
        if (k.next(0) == INT_MAX) continue;
        if (pairs > 0 &&
            !ptx::mbar_wait(q_empty, (pairs - 1) & 1, abort_flag, p.err, ERR_WIN_PRODUCER, patient_ns)) {
          ok = false;
          break;
        }
        ptx::mbar_arrive_expect_tx(q_full, 2 * TILE);
        ++pairs;
#pragma unroll
        for (int b = 0; b < 2; ++b) {
          const int qcol = (k.jj0 + b * hstep) * HD, qrow = (k.qb0 + b * qstep) * BQ;
          ptx::tma_load_3d(sQ + b * TILE, &tm_qkv, q_full, qcol, qrow, k.shard);
          ptx::tma_load_3d(sQ + b * TILE + PANEL, &tm_qkv, q_full, qcol + 64, qrow, k.shard);
        }
        for (int x = k.next(0); ok && x != INT_MAX; x = k.next(x + 1)) {
#pragma unroll
          for (int kv = 0; kv < 2; ++kv) {
            const uint32_t slot = issued % KV_SLOTS;
            if (!ptx::mbar_wait(&kv_empty[slot], ((issued / KV_SLOTS) & 1) ^ 1u, abort_flag, p.err, ERR_WIN_PRODUCER,
                                patient_ns)) {
              ok = false;
              break;
            }
            const int col = kv ? k.vcol : k.kcol;
            uint8_t* dst = sKV + slot * TILE;
            ptx::mbar_arrive_expect_tx(&kv_full[slot], TILE);
            ptx::tma_load_3d(dst, &tm_qkv, &kv_full[slot], col, x * BKV, k.shard);
            ptx::tma_load_3d(dst + PANEL, &tm_qkv, &kv_full[slot], col + 64, x * BKV, k.shard);
            ++issued;
          }
        }
      }
      if (ok) queue.post_end(abort_flag, p.err, ERR_WIN_PRODUCER, patient_ns);
      // drain: every issued copy must land before the CTA exits
      queue.drain(p.err, ERR_WIN_DRAIN, patient_ns);
      volatile int never = 0;
      if (pairs > 0) ptx::mbar_wait(q_full, (pairs - 1) & 1, &never, p.err, ERR_WIN_DRAIN, patient_ns);
      for (uint32_t i = (issued > KV_SLOTS ? issued - KV_SLOTS : 0); i < issued; ++i)
        ptx::mbar_wait(&kv_full[i % KV_SLOTS], (i / KV_SLOTS) & 1, &never, p.err, ERR_WIN_DRAIN, patient_ns);
    }
  } else if (warp == 1) {
    if (ptx::elect_one()) {
      constexpr uint32_t idesc_s = ptx::idesc_f16_f32(BQ, BKV, false, false);
      constexpr uint32_t idesc_o = ptx::idesc_f16_f32(BQ, HD, false, true);
      // Descriptors are formed once; a tile or a k-step is an addition.
      const uint64_t dQ = ptx::sdesc_sw128(ptx::smem_addr(sQ), 16, 1024);
      const uint64_t dKV = ptx::sdesc_sw128(ptx::smem_addr(sKV), 16, 1024);        // rows as they are
      const uint64_t dKVT = ptx::sdesc_sw128(ptx::smem_addr(sKV), PANEL, 1024);    // .. transposed
      auto item_ready = [&](uint32_t i) {
        return ptx::mbar_wait(&kv_full[i % KV_SLOTS], (i / KV_SLOTS) & 1, abort_flag, p.err, ERR_WIN_MMA,
                              patient_ns);
      };
      auto issue_s = [&](int b, int slot) {
        const uint64_t k = ptx::sdesc_at(dKV, slot * TILE);
#pragma unroll
        for (int kk = 0; kk < HD / 16; ++kk)
          ptx::mma_bf16(tmem + 128 * b, ptx::sdesc_at(dQ, b * TILE + kstep(kk, PANEL)), ptx::sdesc_at(k, kstep(kk, PANEL)),
                        idesc_s, kk > 0 ? 1u : 0u);
        ptx::mma_commit(&s_full[b]);
      };
      uint32_t pairs = 0, item = 0;       // item: the next key or value tile of the ring
      uint32_t blk[2] = {0, 0};           // blocks that each tile has finished
      uint32_t outs[2] = {0, 0};          // pairs that each tile took part in
      bool ok = true;
      FwdWork k;
      while (ok && queue.read<false>(k, abort_flag, p.err, ERR_WIN_MMA, patient_ns)) {
        int x = k.next(0);
        if (x == INT_MAX) continue;
        if (!ptx::mbar_wait(q_full, pairs & 1, abort_flag, p.err, ERR_WIN_MMA, patient_ns) || !item_ready(item)) break;
        ++pairs;
        ptx::tc_fence_after();
        // S_b overwrites the P_b of the pair before, whose last P V was issued already: MMAs of one
        // thread run in issue order
        if (k.l0.has(x)) issue_s(0, item % KV_SLOTS);
        if (k.l1.has(x)) issue_s(1, item % KV_SLOTS);
        ptx::mma_commit(&kv_empty[item % KV_SLOTS]);
        int xn = k.next(x + 1);
        if (xn == INT_MAX) ptx::mma_commit(q_empty);
        bool first[2] = {true, true};
        // Per block: P_0 V, S_0 of the next block, P_1 V, S_1 of the next, each only where the tile has
        // that block.
        for (; ok && x != INT_MAX; item += 2) {
          const uint32_t iv = item + 1, ik = item + 2;
          if (!item_ready(iv)) {
            ok = false;
            break;
          }
          if (total < p.N && x * BKV + BKV > total) {
            // Rows behind the last sequence may hold anything; their P is 0, but 0 * inf is not: zero their
            // V rows (whole 128-byte rows, so the swizzle does not matter).
            uint8_t* v = sKV + (iv % KV_SLOTS) * TILE;
            for (int r = max(total - x * BKV, 0); r < BKV; ++r)
#pragma unroll
              for (int c = 0; c < 8; ++c) {
                *reinterpret_cast<uint4*>(v + r * 128 + c * 16) = make_uint4(0u, 0u, 0u, 0u);
                *reinterpret_cast<uint4*>(v + PANEL + r * 128 + c * 16) = make_uint4(0u, 0u, 0u, 0u);
              }
            ptx::fence_proxy_async_smem();
          }
          const int xnn = xn == INT_MAX ? INT_MAX : k.next(xn + 1);
          bool k_next = false;
#pragma unroll
          for (int b = 0; b < 2; ++b) {
            const KeyBlocks& l = b ? k.l1 : k.l0;
            if (l.has(x)) {
              if (!ptx::mbar_wait(&p_half[b], blk[b] & 1, abort_flag, p.err, ERR_WIN_MMA, patient_ns) ||
                  (first[b] && outs[b] > 0 &&
                   !ptx::mbar_wait(&o_empty[b], (outs[b] - 1) & 1, abort_flag, p.err, ERR_WIN_MMA, patient_ns))) {
                ok = false;
                break;
              }
              ptx::tc_fence_after();
              const uint64_t v = ptx::sdesc_at(dKVT, (iv % KV_SLOTS) * TILE);
#pragma unroll
              for (int half = 1; half >= 0; --half) {
                if (half == 0) {
                  if (!ptx::mbar_wait(&p_full[b], blk[b] & 1, abort_flag, p.err, ERR_WIN_MMA, patient_ns)) {
                    ok = false;
                    break;
                  }
                  ptx::tc_fence_after();
                }
#pragma unroll
                for (int kk = 4 * half; kk < 4 * half + 4; ++kk)
                  ptx::mma_f16_ts(tmem + 256 + 128 * b, tmem + 128 * b + 64 + kk * 8, ptx::sdesc_at(v, kk * 2048),
                                  idesc_o, (!first[b] || kk != 4) ? 1u : 0u);
              }
              if (!ok) break;
              first[b] = false;
              ++blk[b];
              if (l.from(x + 1) == INT_MAX) {
                ptx::mma_commit(&o_full[b]);
                ++outs[b];
              }
            }
            if (xn != INT_MAX && l.has(xn)) {
              if (!k_next) {
                if (!item_ready(ik)) {
                  ok = false;
                  break;
                }
                ptx::tc_fence_after();
                k_next = true;
              }
              issue_s(b, ik % KV_SLOTS);
            }
          }
          if (!ok) break;
          ptx::mma_commit(&kv_empty[iv % KV_SLOTS]);
          if (k_next) ptx::mma_commit(&kv_empty[ik % KV_SLOTS]);
          if (xn != INT_MAX && xnn == INT_MAX) ptx::mma_commit(q_empty);  // the last block's S were issued
          x = xn;
          xn = xnn;
        }
      }
      ptx::mma_commit(mma_done);
      volatile int never = 0;
      ptx::mbar_wait(mma_done, 0, &never, p.err, ERR_WIN_DRAIN, patient_ns);
    }
  } else {
    // ------------------------------------------------------- softmax rows
    // Warps 2-5 own tile 0, warps 6-9 tile 1; a warp reads the TMEM lanes of its rank within a
    // warpgroup (warp & 3), one query row per thread.
    const int b = (warp - 2) >> 2;
    const uint32_t lane_base = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t tSb = tmem + 128 * b + lane_base, tOb = tSb + 256;
    const float sl2 = NEG ? -p.scale_log2 : p.scale_log2;  // >= 0 once S is negated under a negative scale
    uint32_t blk = 0, outs = 0;  // blocks, pairs that this tile has finished
    bool ok = true;
    while (ok) {
      int q, st, shard, jj;
      KeyBlocks l;
      {
        FwdWork k;
        if (!queue.read<true>(k, abort_flag, p.err, ERR_WIN_SOFTMAX, patient_ns)) break;
        q = (k.qb0 + b * qstep) * BQ + (warp & 3) * 32 + lane;
        shard = k.shard;
        jj = k.jj0 + b * hstep;
        l = b ? k.l1 : k.l0;
        st = b ? k.st1 : k.st0;
      }
      const bool alive = q < total;
      if (st < 0) st = alive ? span_of(p, q).x : 0;
      const int wlo = max(st, q - p.W + 1);                 // the window's first key
      const int shi = p.S > 0 ? min(st + p.S - 1, q) : -1;  // the last visible sink
      // m is the row's reference maximum (log2 domain).  It is raised only when a
      // block's maximum exceeds it by more than kLazyRescale, so most blocks skip the
      // O rescale; P is then at most 2^kLazyRescale, well inside fp16.
      float m = kNoMax, lsum = 0.0f;
      bool first = true;
      for (int x = l.from(0); x != INT_MAX; x = l.from(x + 1)) {
        const int kv0 = x * BKV;
        const int w0 = wlo - kv0, w1 = q - kv0, s0 = st - kv0, s1 = shi - kv0;  // visible columns of this row
        // Blocks at an edge have code of their own, and as little of it as it can be: one set of code with a
        // branch for each 32 columns took 2800 us where the two take 2535, and masked copies of all of it for the
        // edges 431 instead of 400 (packed prefill, N 15937, W 1024).
        // Known before the scores are: whether every row of the warp sees all 128 columns; if not, the columns that
        // this row sees, and the runs of 32 of which the rows see all or nothing.
        const bool full = !alive || (w0 <= 0 && w1 >= BKV - 1) || (s0 <= 0 && s1 >= BKV - 1);
        const bool plain = !NEG && __all_sync(0xffffffffu, full);
        uint32_t bits[4], all = 0, any = 0;
        if (!plain) {
#pragma unroll
          for (int h = 0; h < 4; ++h) {
            const int c = h * 32;
            bits[h] = alive ? span_bits(w0 - c, w1 - c) | span_bits(s0 - c, s1 - c) : 0xffffffffu;
            all |= __all_sync(0xffffffffu, bits[h] == 0xffffffffu) ? 1u << h : 0u;
            any |= __any_sync(0xffffffffu, bits[h] != 0u) ? 1u << h : 0u;
          }
        }
        if (!warp_wait(&s_full[b], blk & 1, abort_flag, p.err, ERR_WIN_SOFTMAX, patient_ns)) {
          ok = false;
          break;
        }
        ptx::tc_fence_after();
        float m_new, alpha;
        uint64_t rs2[2] = {f2_pack(0.0f, 0.0f), f2_pack(0.0f, 0.0f)};
        auto softmax = [&](auto whole) {
          constexpr bool PLAIN = decltype(whole)::value;  // every row sees all 128 keys
          // Pass 1: the block's row maximum.  The last 64 scores stay in registers for pass 2, the first 64 are read
          // once more (all 128 in registers spill).  Each load runs while the scores before it are worked on.
          float mx4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
          auto row_max = [&](uint32_t (&r)[32], int h) {
            if (NEG) {
              max32_neg(r, bits[h], mx4);
            } else if (PLAIN || ((any >> h) & 1u)) {
              if (!PLAIN && !((all >> h) & 1u)) mask32(r, bits[h]);
              max32(r, mx4);
            }
          };
          uint32_t lo[32], hi[2][32];
          ptx::tmem_ld32(tSb, lo);
          ptx::tmem_ld_wait32(lo);
          {
            uint32_t lo1[32];
            ptx::tmem_ld32(tSb + 32, lo1);
            row_max(lo, 0);
            ptx::tmem_ld_wait32(lo1);
            ptx::tmem_ld32(tSb + 64, hi[0]);
            ptx::tmem_ld32(tSb + 96, hi[1]);
            row_max(lo1, 1);
          }
          ptx::tmem_ld_wait32(hi[0]);
          ptx::tmem_ld_wait32(hi[1]);
          ptx::tmem_ld32(tSb, lo);
          row_max(hi[0], 2);
          row_max(hi[1], 3);
          // a row that sees nothing here keeps its reference
          const float top = max3f(mx4[0], mx4[1], fmaxf(mx4[2], mx4[3]));
          const float mx = top == -INFINITY ? kNoMax : top * sl2;
          m_new = (mx > m + kLazyRescale) ? mx : m;
          alpha = ptx::exp2_approx(m - m_new);  // 0 on the row's first keys, 1 when m stays
          if (!first && __any_sync(0xffffffffu, m_new != m)) {
            // O_b is idle: the P V of its previous block finished before this S_b was committed.
#pragma unroll 1
            for (int c = 0; c < 4; ++c) {
              uint32_t o[32];
              ptx::tmem_ld32(tOb + c * 32, o);
              ptx::tmem_ld_wait();
#pragma unroll
              for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
              ptx::tmem_st32(tOb + c * 32, o);
            }
          }
          // Pass 2: P = 2^(S scale - m), 32 columns at a time, written as fp16 pairs over S's last 64 columns (in
          // registers by now), those of keys 64-127 first: their half of P V runs while the other half is formed
          // (N 16384, 64 heads, full causal: 2535 us, 1735 TFLOP/s; P handed over whole 2750).
          const float neg_m = -m_new;
          auto prob = [&](uint32_t (&r)[32], int h) {
            uint32_t wd[16];
            if (NEG) {
              exp32_neg(r, bits[h], sl2, neg_m, rs2, wd);
            } else if (PLAIN || ((any >> h) & 1u)) {
              if (!PLAIN && h < 2 && !((all >> h) & 1u)) mask32(r, bits[h]);  // read once more
              exp32(r, sl2, neg_m, rs2, wd);
            } else {
#pragma unroll
              for (int e = 0; e < 16; ++e) wd[e] = 0u;
            }
            ptx::tmem_st16(tSb + 64 + h * 16, wd);
          };
          auto arrive = [&](uint64_t* bar) {
            ptx::tmem_st_wait();
            ptx::tc_fence_before();
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(bar);
          };
          prob(hi[0], 2);
          prob(hi[1], 3);
          arrive(&p_half[b]);
          ptx::tmem_ld_wait32(lo);
          ptx::tmem_ld32(tSb + 32, hi[0]);
          prob(lo, 0);
          ptx::tmem_ld_wait32(hi[0]);
          prob(hi[0], 1);
          arrive(&p_full[b]);
        };
        if (plain)
          softmax(std::true_type());
        else
          softmax(std::false_type());
        float rs4[4];
        f2_unpack(rs2[0], rs4[0], rs4[1]);
        f2_unpack(rs2[1], rs4[2], rs4[3]);
        lsum = fmaf(lsum, alpha, (rs4[0] + rs4[1]) + (rs4[2] + rs4[3]));
        m = m_new;
        first = false;
        ++blk;
      }
      uint16_t* orow = p.O + (static_cast<int64_t>(shard) * p.N + q) * p.dt + static_cast<int64_t>(jj) * HD;
      float* lrow = p.lse + (static_cast<int64_t>(shard) * p.hpr + jj) * p.N + q;
      if (!first && ok) {
        if (!warp_wait(&o_full[b], outs & 1, abort_flag, p.err, ERR_WIN_SOFTMAX, patient_ns)) {
          ok = false;
          break;
        }
        ++outs;
        ptx::tc_fence_after();
        const float inv = 1.0f / lsum;
        const uint64_t inv_l = f2_pack(inv, inv);
        uint64_t odd = 0;  // NaN once an element is not finite
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          uint32_t o[32];
          ptx::tmem_ld32(tOb + c * 32, o);
          ptx::tmem_ld_wait();
          if (c == 3) {  // the next pair's P V may overwrite O_b
            ptx::tc_fence_before();
            ptx::mbar_arrive(&o_empty[b]);
          }
          uint32_t v[16];
#pragma unroll
          for (int e = 0; e < 32; e += 2) {
            const uint64_t x2 = f2_pack(__uint_as_float(o[e]), __uint_as_float(o[e + 1]));
            odd = f2_fma(x2, 0, odd);
            float x0, x1;
            f2_unpack(f2_mul(x2, inv_l), x0, x1);
            v[e >> 1] = pack_bf16x2(x0, x1);
          }
          if (alive && p.wide) {  // 32 bytes a store: whole sectors
            st_global_32b(orow + c * 32, v);
            st_global_32b(orow + c * 32 + 16, v + 8);
          } else if (alive) {
#pragma unroll
            for (int e = 0; e < 16; e += 4)
              *reinterpret_cast<uint4*>(orow + c * 32 + 2 * e) = make_uint4(v[e], v[e + 1], v[e + 2], v[e + 3]);
          }
        }
        if (alive) *lrow = (m + __log2f(lsum)) * kLn2;
        float o0, o1;
        f2_unpack(odd, o0, o1);
        uint32_t again =
            __ballot_sync(0xffffffffu, alive && !(o0 == 0.0f && o1 == 0.0f && lsum > 0.0f && lsum < INFINITY));
        while (again) {
          const int r = __ffs(again) - 1;
          again &= again - 1;
          const int qr = __shfl_sync(0xffffffffu, q, r), sr = __shfl_sync(0xffffffffu, st, r);
          __syncwarp();
          const int gcol = (jj / p.Gs) * HD;
          slow_row(p, shard, jj * HD, static_cast<int>(p.kcol0) + gcol, static_cast<int>(p.vcol0) + gcol, qr, sr,
                   orow + (r - lane) * p.dt, lrow + (r - lane));
        }
      }
      if (p.zero_pad && q < p.N && !alive) {
#pragma unroll
        for (int c = 0; c < HD; c += 8) *reinterpret_cast<uint4*>(orow + c) = make_uint4(0u, 0u, 0u, 0u);
        *lrow = 0.0f;
      }
    }
  }

  ptx::tc_fence_before();
  __syncwarp();  // lane-0 roles rejoin their warp: bar.sync needs converged warps
  __syncthreads();
  if (warp == 1) {
    __syncwarp();
    ptx::tc_fence_after();
    ptx::tmem_dealloc(tmem, 512);
  }
}

// ------------------------------------------------------------------ backward
//
// The two kernels of attention.cu over the visible blocks: dK / dV per 128-key block with the keys on
// the TMEM lanes, looping over 64-query blocks of the group's heads; dQ per 128-query block over
// 64-key blocks.  The scores of a block are formed again from the saved lse.  A hidden pair's P and
// dS are selected to 0, whatever its operands hold.
constexpr int P_EXP = 13;              // P 2^13: at most 1 but for lse's error, which has 2^2 of room
constexpr int BWD_THREADS = 320;       // TMA warp, MMA warp, eight compute warps
constexpr int BWD_STAGES = 4;
constexpr int DKV_SMEM = 1024 + 2 * TILE + BWD_STAGES * (2 * TILE64 + 512) + 256 + QUEUE_SMEM;
constexpr int DQ_THREADS = 448;        // .. and four output warps
constexpr int DQ_STAGES = 4;
// The next block of queries is asked for this many steps before the last loads, as its D has to be there when
// the block before ends: 0 and 3 steps took 651 and 636 us (N 16384, W 1024, seven sequences), 6 take 632.
constexpr int DQ_AHEAD = 6;
constexpr int DQ_SMEM = 1024 + 2 * TILE + DQ_STAGES * 2 * TILE64 + 256 + QUEUE_SMEM + 2 * (128 + 4) * 4;
// With 1 KB of the system's the block stays within the 196 KB split of an SM's memory, so 60 KB of it cache the output
// warps' loads; one KB more takes the 228 KB split, 672 us where this takes 645 (N 16384, W 1024, seven sequences).
static_assert(DQ_SMEM + 1024 <= 196 * 1024, "the next larger shared memory split");

// The largest sum|v| of a key block: in dV, 64 blocks a row, until the dK / dV kernel, behind dQ's, writes that.
__device__ __forceinline__ float* value_bound(const WinArgs& p, int shard, int vcol, int kb) {
  return reinterpret_cast<float*>(p.dQKV + (static_cast<int64_t>(shard) * p.N + kb / 64) * p.row_w + vcol) + kb % 64;
}
// The largest B of the query heads that share head jj's KV head, as the bits of a float that is not negative: in the
// place of D of the first such head's row 0, a row that sees one key, whose D has no use.
__device__ __forceinline__ unsigned* row_bound(const WinArgs& p, int shard, int jj) {
  return reinterpret_cast<unsigned*>(p.Dvec + (static_cast<int64_t>(shard) * p.hpr + jj / p.Gs * p.Gs) * p.N);
}
// e of a bound B, and 2^e.
__device__ __forceinline__ int ds_exponent(float bound) {
  const int x = static_cast<int>(__float_as_uint(bound) >> 23) - 127;  // floor(log2 B), -127 for 0
  return max(-30, min(P_EXP - x, 64));  // finite fp16 operands: B is 0 or 2^-48 .. 2^39
}
__device__ __forceinline__ float power2(int e) { return __uint_as_float(static_cast<uint32_t>(e + 127) << 23); }

// The first 64-query block beyond the window's reach of key block kb: the block's own CTA takes the
// queries before it, the far CTAs those from it on (only sinks are seen from there).
__device__ __forceinline__ int reach64(const WinArgs& p, int kb) { return (kb * BKV + BKV - 1 + p.W + 63) >> 6; }

// A query that sees its own key only: P = 1, and dP - D, which is 0, would leave the rounding of O to bf16 in D
// (2.4e-3 of the whole gradient under a window of 1).  Its dS is 0.
__device__ __forceinline__ bool sees_one(const WinArgs& p, int q, int st) { return q == st || (p.W == 1 && p.S == 0); }

// P and dS of one key row (or query row) and 32 scores: p = 2^(s sl2 + nl), d = p (dp up + nd), packed
// fp16; up and the powers of two in nd (and nl) make them d 2^e (and p 2^13).  ROWQ: nl, nd are the row's (dQ);
// else nlv, ndv hold one per column (dK / dV, shared memory).  Unless plain, p is 0 outside bits and d outside dbits.
template <bool ROWQ>
__device__ __forceinline__ void p_ds32(const uint32_t (&s)[32], const uint32_t (&dp)[32], float sl2, float nl, float nd,
                                       float up, const float4* nlv, const float4* ndv, bool plain, uint32_t bits,
                                       uint32_t dbits, uint32_t (&wp)[16], uint32_t (&wds)[16]) {
  const uint64_t sl2x2 = f2_pack(sl2, sl2), nl2 = f2_pack(nl, nl), nd2 = f2_pack(nd, nd), up2 = f2_pack(up, up);
#pragma unroll
  for (int e4 = 0; e4 < 8; ++e4) {
    float4 L4, D4;
    if (!ROWQ) {
      L4 = nlv[e4];
      D4 = ndv[e4];
    }
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int e = 4 * e4 + 2 * u;
      const uint64_t a = ROWQ ? nl2 : (u ? f2_pack(L4.z, L4.w) : f2_pack(L4.x, L4.y));
      const uint64_t d = ROWQ ? nd2 : (u ? f2_pack(D4.z, D4.w) : f2_pack(D4.x, D4.y));
      float x0, x1;
      f2_unpack(f2_fma(f2_pack(__uint_as_float(s[e]), __uint_as_float(s[e + 1])), sl2x2, a), x0, x1);
      float p0 = ptx::exp2_approx(x0), p1 = ptx::exp2_approx(x1);
      float d0, d1;
      f2_unpack(f2_mul(f2_pack(p0, p1), f2_fma(f2_pack(__uint_as_float(dp[e]), __uint_as_float(dp[e + 1])), up2, d)), d0,
                d1);
      if (!plain) {
        if (!ROWQ) {
          p0 = (bits >> e) & 1u ? p0 : 0.0f;
          p1 = (bits >> (e + 1)) & 1u ? p1 : 0.0f;
        }
        d0 = (dbits >> e) & 1u ? d0 : 0.0f;
        d1 = (dbits >> (e + 1)) & 1u ? d1 : 0.0f;
      }
      if (!ROWQ) wp[2 * e4 + u] = pack_f16x2(p0, p1);
      wds[2 * e4 + u] = pack_f16x2(d0, d1);
    }
  }
}

// What the rows of a warp see of their 32 columns (formed before the wait for the scores).
enum Sight : int { SEES_NONE, SEES_SOME, SEES_ALL };
__device__ __forceinline__ Sight sight_of(uint32_t bits) {
  if (!__any_sync(0xffffffffu, bits != 0u)) return SEES_NONE;
  return __all_sync(0xffffffffu, bits == 0xffffffffu) ? SEES_ALL : SEES_SOME;
}

// One thread's 32 scores and dP of a step in TMEM to P and dS, written over their first 16 columns (P only
// where it is an operand: dK / dV).  Columns that no row of the warp sees become 0 without the arithmetic.
template <bool ROWQ>
__device__ __forceinline__ void p_ds_step(uint32_t tS, uint32_t tdP, float sl2, float nl, float nd, float up,
                                          const float4* nlv, const float4* ndv, uint32_t bits, uint32_t dbits,
                                          Sight sight) {
  uint32_t wp[16], wds[16];
  if (sight == SEES_NONE) {
#pragma unroll
    for (int e = 0; e < 16; ++e) wp[e] = wds[e] = 0u;
  } else {
    uint32_t s[32], dp[32];
    ptx::tmem_ld32(tS, s);
    ptx::tmem_ld32(tdP, dp);
    ptx::tmem_ld_wait();
    if (sight == SEES_ALL) p_ds32<ROWQ>(s, dp, sl2, nl, nd, up, nlv, ndv, true, 0u, 0u, wp, wds);
    else p_ds32<ROWQ>(s, dp, sl2, nl, nd, up, nlv, ndv, false, bits, dbits, wp, wds);
  }
  if (ROWQ) {
    ptx::tmem_st16(tS, wds);
  } else {
    ptx::tmem_st16(tS, wp);
    ptx::tmem_st16(tdP, wds);
  }
}

// fp32 dV, dK [2][128] of sink `idx` of its sequence for KV head kvh, from the far queries of `chunk`, or, at
// nch + its first far chunk, from the queries within its block's reach.  A chunk has far queries of one
// sequence only, so rows of different sequences never meet.
__device__ __forceinline__ float* far_row(const WinArgs& p, int kvh, int chunk, int idx) {
  return p.far + ((static_cast<int64_t>(kvh) * 2 * p.nch + chunk) * p.S + idx) * 2 * HD;
}

// 16 values of 16 bits to a 16-byte (wide: 32-byte) aligned address.
__device__ __forceinline__ void store_16(uint16_t* dst, const uint32_t (&v)[8], int wide) {
  if (wide) {
    st_global_32b(dst, v);
  } else {
    *reinterpret_cast<uint4*>(dst) = make_uint4(v[0], v[1], v[2], v[3]);
    *reinterpret_cast<uint4*>(dst + 8) = make_uint4(v[4], v[5], v[6], v[7]);
  }
}

__device__ __forceinline__ void zero_row128(uint8_t* row) {
#pragma unroll
  for (int c = 0; c < 8; ++c) *reinterpret_cast<uint4*>(row + c * 16) = make_uint4(0u, 0u, 0u, 0u);
}

// One key block of one KV head, and the 64-query blocks [q_first, q_end) of its group's heads that it
// meets.  The first nfar works are far ones: the queries of one chunk beyond the reach of one sink
// block of the sequence (far_st: its first row) that the chunk's first row belongs to; without queries
// when the chunk, the sink or the queries are missing.
struct DkvWork {
  int far, kvh, shard, jl, kb, q_first, q_end, chunk, far_st, kcol, vcol;
  int st, en;  // the sequence of the block's rows, -1: not one for all rows
  int e;       // dS 2^e
  DkvWork() = default;
  __device__ DkvWork(const WinArgs& p, int w, int total) {
    far = w < p.nfar;
    if (!far) w -= p.nfar;
    kvh = w % p.Hkv;
    const int rest = w / p.Hkv;
    shard = kvh / p.kv_t;
    jl = kvh - shard * p.kv_t;
    kcol = static_cast<int>(p.kcol0) + jl * HD;
    vcol = static_cast<int>(p.vcol0) + jl * HD;
    chunk = 0;
    far_st = -1;
    if (far) {
      chunk = rest / p.nsb;
      const int r0 = chunk * p.C;
      const int2 sp = span_of(p, r0);
      far_st = sp.x;
      kb = sp.x / BKV + (rest - chunk * p.nsb);
      q_first = max(r0 / 64, reach64(p, kb));
      q_end = min((r0 + p.C) / 64, (sp.y + 63) / 64);
      if (sp.y <= r0 || kb * BKV >= sp.x + p.S) q_end = q_first;
    } else {
      kb = rest;
      q_first = 2 * kb;
      const int last = min(kb * BKV + BKV - 1, total - 1);  // only the last row's sequence goes on behind the block
      q_end = last < kb * BKV ? q_first : min(reach64(p, kb), (span_of(p, last).y + 63) / 64);
      chunk = p.nch + reach64(p, kb) * 64 / max(p.C, 1);
    }
    q_end = max(q_end, q_first);
    st = common_begin(p, kb * BKV, BKV, total);
    en = span_of(p, kb * BKV).y;
    e = ds_exponent(__uint_as_float(*row_bound(p, shard, jl * p.Gs)));
  }
  __device__ int nq() const { return q_end - q_first; }
};

// Persistent, as the forward: the next block's K and V load while the last P, dS and the output of the
// one before are worked on.  Counters that give barrier phases run on over the blocks.
__global__ void __launch_bounds__(BWD_THREADS, 1)
    window_dkv_kernel(const __grid_constant__ CUtensorMap tm_qkv, const __grid_constant__ CUtensorMap tm_do,
                      const WinArgs p) {
  extern __shared__ uint8_t dsmem[];
  const uint32_t pad = (1024u - (ptx::smem_addr(dsmem) & 1023u)) & 1023u;
  uint8_t* base = dsmem + pad;
  uint8_t* sK = base;
  uint8_t* sV = base + TILE;
  uint8_t* sQd = base + 2 * TILE;  // stage s: Q_n at s * 2 TILE64, dO_n after it
  float* sLD = reinterpret_cast<float*>(base + 2 * TILE + BWD_STAGES * 2 * TILE64);  // stage s: -lse2[64], -D[64]
  uint64_t* bars = reinterpret_cast<uint64_t*>(base + 2 * TILE + BWD_STAGES * (2 * TILE64 + 512));
  uint64_t* kv_full = bars + 0;
  uint64_t* kv_empty = bars + 1;                   // the block's last S^T, dP^T read K and V
  uint64_t* qd_full = bars + 2;                    // [BWD_STAGES] TMA bytes + 32 lse/D writers
  uint64_t* qd_empty = bars + 2 + BWD_STAGES;      // [BWD_STAGES]
  uint64_t* st_full = bars + 2 + 2 * BWD_STAGES;   // [2] S^T, dP^T of a step in TMEM
  uint64_t* pds_full = bars + 4 + 2 * BWD_STAGES;  // [2] P^T, dS^T written
  uint64_t* acc_full = bars + 6 + 2 * BWD_STAGES;  // dV, dK of the block complete
  uint64_t* acc_empty = bars + 7 + 2 * BWD_STAGES; // .. and read
  uint64_t* mma_done = bars + 8 + 2 * BWD_STAGES;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 9 + 2 * BWD_STAGES);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  WorkQueue<DkvWork, 9> queue(reinterpret_cast<uint8_t*>(bars) + 256);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    ptx::mbar_init(kv_full, 1);
    ptx::mbar_init(kv_empty, 1);
    for (int s = 0; s < BWD_STAGES; ++s) {
      ptx::mbar_init(&qd_full[s], 33);
      ptx::mbar_init(&qd_empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      ptx::mbar_init(&st_full[b], 1);
      ptx::mbar_init(&pds_full[b], 8);
    }
    ptx::mbar_init(acc_full, 1);
    ptx::mbar_init(acc_empty, 256);
    ptx::mbar_init(mma_done, 1);
    queue.init();
    *abort_flag = 0;
    ptx::fence_mbar_init();
  }
  if (warp == 1) {
    ptx::tmem_alloc(tmem_slot, 512);
    ptx::tmem_relinquish();
  }
  ptx::tc_fence_before();
  __syncwarp();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  ptx::griddep_wait();
  ptx::griddep_launch_dependents();
  const int total = total_rows(p);
  // TMEM columns: S^T_0 | S^T_1 (64 each) | dP^T_0 | dP^T_1 (64 each) | dV (128) | dK (128).
  const uint32_t tdV = tmem + 256, tdK = tmem + 384;

  if (warp == 0) {
    // Producer warp: lane 0 issues the tile copies, all 32 lanes stage lse2 / D.
    if (lane == 0) {
      ptx::tma_prefetch_desc(&tm_qkv);
      ptx::tma_prefetch_desc(&tm_do);
    }
    uint32_t issued = 0, blocks = 0;
    bool ok = true;
    for (int w = blockIdx.x; ok && w >= 0;) {
      const int now = w;
      auto advance = [&]() {  // lane 0 asks, every lane gets the answer
        int nx = -1;
        if (lane == 0) nx = queue.next(abort_flag, p.err, ERR_WIN_PRODUCER, p.timeout_ns);
        w = __shfl_sync(0xffffffffu, nx, 0);
      };
      const DkvWork k(p, now, total);
      const int nloop = k.nq() * p.Gs;
      if (lane == 0) ok = queue.post(k, abort_flag, p.err, ERR_WIN_PRODUCER, p.timeout_ns);
      ok = __shfl_sync(0xffffffffu, ok, 0);
      if (!ok) break;
      if (nloop == 0) {
        advance();
        continue;
      }
      if (lane == 0) {
        ok = blocks == 0 ||
             ptx::mbar_wait(kv_empty, (blocks - 1) & 1, abort_flag, p.err, ERR_WIN_PRODUCER, p.timeout_ns);
        if (ok) {
          ptx::mbar_arrive_expect_tx(kv_full, 2 * TILE);
          tma_tile128(sK, &tm_qkv, kv_full, k.kcol, k.kb * BKV, k.shard);
          tma_tile128(sV, &tm_qkv, kv_full, k.vcol, k.kb * BKV, k.shard);
        }
      }
      ok = __shfl_sync(0xffffffffu, ok, 0);
      if (!ok) break;
      ++blocks;
      // A step's lse and D are on their way while the step before waits for its slot: loaded in their own step they
      // cost each one a trip to memory, 700 of 1,700 cycles in which the MMAs waited for this warp.
      int qi = k.q_first, qh = k.jl * p.Gs;
      float nl[2], nd[2];  // of the queries qi * 64 + lane, + 32; negated: the compute warps add them
      auto load_row = [&]() {
        const int64_t vec = (static_cast<int64_t>(k.shard) * p.hpr + qh) * p.N;
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int q = qi * 64 + lane + 32 * e;
          nl[e] = q < p.N ? p.lse[vec + q] : 0.0f;
          nd[e] = q < p.N && q > 0 ? p.Dvec[vec + q] : 0.0f;  // row 0: row_bound()
        }
      };
      load_row();
      const float up = power2(k.e - P_EXP);
      for (int n = 0; n < nloop; ++n, ++issued) {
        const uint32_t slot = issued % BWD_STAGES;
        const int q0 = qi * 64, qcol = qh * HD;
        const float l0 = nl[0], l1 = nl[1], d0 = nd[0], d1 = nd[1];
        if (++qi == k.q_end) {
          qi = k.q_first;
          ++qh;
        }
        if (n + 1 < nloop) load_row();
        if (lane == 0)
          ok = ptx::mbar_wait(&qd_empty[slot], ((issued / BWD_STAGES) & 1) ^ 1u, abort_flag, p.err, ERR_WIN_PRODUCER,
                              p.timeout_ns);
        ok = __shfl_sync(0xffffffffu, ok, 0);
        if (!ok) break;
        __syncwarp();
        uint8_t* dst = sQd + slot * 2 * TILE64;
        if (lane == 0) {
          ptx::mbar_arrive_expect_tx(&qd_full[slot], 2 * TILE64);
          tma_tile64(dst, &tm_qkv, &qd_full[slot], qcol, q0, k.shard);
          tma_tile64(dst + TILE64, &tm_do, &qd_full[slot], qcol, q0, k.shard);
        }
        float* ld = sLD + slot * 128 + lane;
        ld[0] = P_EXP - l0 * kLog2e;
        ld[32] = P_EXP - l1 * kLog2e;
        ld[64] = -d0 * up;
        ld[96] = -d1 * up;
        ptx::mbar_arrive(&qd_full[slot]);
      }
      if (ok) advance();
    }
    __syncwarp();
    if (lane == 0) {
      if (ok) queue.post_end(abort_flag, p.err, ERR_WIN_PRODUCER, p.timeout_ns);
      queue.drain(p.err, ERR_WIN_DRAIN, p.timeout_ns);
      volatile int never = 0;
      if (blocks > 0) ptx::mbar_wait(kv_full, (blocks - 1) & 1, &never, p.err, ERR_WIN_DRAIN, p.timeout_ns);
      for (uint32_t n = (issued > BWD_STAGES ? issued - BWD_STAGES : 0); n < issued; ++n)
        ptx::mbar_wait(&qd_full[n % BWD_STAGES], (n / BWD_STAGES) & 1, &never, p.err, ERR_WIN_DRAIN, p.timeout_ns);
    }
  } else if (warp == 1) {
    if (ptx::elect_one()) {
      constexpr uint32_t idesc_st = ptx::idesc_f16_f32(128, 64, false, false);   // S^T, dP^T
      constexpr uint32_t idesc_acc = ptx::idesc_f16_f32(128, 128, false, true);  // dV, dK
      // Descriptors are formed once; a tile or a k-step is an addition.
      const uint64_t dK = ptx::sdesc_sw128(ptx::smem_addr(sK), 16, 1024);
      const uint64_t dV = ptx::sdesc_sw128(ptx::smem_addr(sV), 16, 1024);
      const uint64_t dQd = ptx::sdesc_sw128(ptx::smem_addr(sQd), 16, 1024);         // rows as they are
      const uint64_t dQdT = ptx::sdesc_sw128(ptx::smem_addr(sQd), PANEL64, 1024);   // .. transposed
      auto issue_st = [&](uint32_t n) {
        const uint32_t slot = n % BWD_STAGES, b = n & 1;
        if (!ptx::mbar_wait(&qd_full[slot], (n / BWD_STAGES) & 1, abort_flag, p.err, ERR_WIN_MMA, p.timeout_ns))
          return false;
        ptx::tc_fence_after();
        const uint64_t q = ptx::sdesc_at(dQd, slot * 2 * TILE64);
#pragma unroll
        for (int kk = 0; kk < 8; ++kk)
          ptx::mma_bf16(tmem + 64 * b, ptx::sdesc_at(dK, kstep(kk, PANEL)), ptx::sdesc_at(q, kstep(kk, PANEL64)), idesc_st,
                        kk > 0 ? 1u : 0u);
#pragma unroll
        for (int kk = 0; kk < 8; ++kk)
          ptx::mma_bf16(tmem + 128 + 64 * b, ptx::sdesc_at(dV, kstep(kk, PANEL)),
                        ptx::sdesc_at(q, TILE64 + kstep(kk, PANEL64)), idesc_st, kk > 0 ? 1u : 0u);
        ptx::mma_commit(&st_full[b]);
        return true;
      };
      uint32_t n = 0, blocks = 0;  // steps, blocks so far
      bool ok = true;
      DkvWork k;
      while (ok && queue.read<false>(k, abort_flag, p.err, ERR_WIN_MMA, p.timeout_ns)) {
        const int nloop = k.nq() * p.Gs;
        if (nloop == 0) continue;
        ok = ptx::mbar_wait(kv_full, blocks & 1, abort_flag, p.err, ERR_WIN_MMA, p.timeout_ns) && issue_st(n);
        if (ok && nloop == 1) ptx::mma_commit(kv_empty);
        // Step i+1's S^T / dP^T go in before step i's dV / dK: the tensor pipe works on them
        // while the compute warps form P^T_i and dS^T_i.  Buffer (n+1) & 1 was last read by
        // the dV / dK MMAs of step n-1, issued (and so executed) before.
        for (int i = 0; ok && i < nloop; ++i, ++n) {
          if (i + 1 < nloop) {
            if (!issue_st(n + 1)) {
              ok = false;
              break;
            }
            if (i + 2 == nloop) ptx::mma_commit(kv_empty);
          }
          const uint32_t b = n & 1, slot = n % BWD_STAGES;
          if (!ptx::mbar_wait(&pds_full[b], (n >> 1) & 1, abort_flag, p.err, ERR_WIN_MMA, p.timeout_ns) ||
              (i == 0 && blocks > 0 &&
               !ptx::mbar_wait(acc_empty, (blocks - 1) & 1, abort_flag, p.err, ERR_WIN_MMA, p.timeout_ns))) {
            ok = false;
            break;
          }
          ptx::tc_fence_after();
          const uint64_t q = ptx::sdesc_at(dQdT, slot * 2 * TILE64);
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            ptx::mma_f16_ts(tdV, tmem + 64 * b + half_split_col(kk), ptx::sdesc_at(q, TILE64 + kk * 2048), idesc_acc,
                            (i > 0 || kk > 0) ? 1u : 0u);
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            ptx::mma_f16_ts(tdK, tmem + 128 + 64 * b + half_split_col(kk), ptx::sdesc_at(q, kk * 2048), idesc_acc,
                            (i > 0 || kk > 0) ? 1u : 0u);
          ptx::mma_commit(&qd_empty[slot]);
        }
        if (!ok) break;
        ptx::mma_commit(acc_full);
        ++blocks;
      }
      ptx::mma_commit(mma_done);
      volatile int never = 0;
      ptx::mbar_wait(mma_done, 0, &never, p.err, ERR_WIN_DRAIN, p.timeout_ns);
    }
  } else {
    // Compute warps: lane quarter warp & 3 (key rows), column half h of each 64-query block.
    const int quad = warp & 3, h = (warp - 2) >> 2;
    const int row = quad * 32 + lane;
    const uint32_t lane_base = static_cast<uint32_t>(quad * 32) << 16;
    uint32_t n = 0, blocks = 0;
    bool ok = true;
    DkvWork k;
    while (ok && queue.read<true>(k, abort_flag, p.err, ERR_WIN_SOFTMAX, p.timeout_ns)) {
      const int nloop = k.nq() * p.Gs;
      if (k.far && nloop == 0) continue;
      const int kv = k.kb * BKV + row;
      // this key is seen by the queries kv .. qmax
      const bool alive = kv < total;
      const int2 sp = !alive ? make_int2(0, 0) : k.st >= 0 ? make_int2(k.st, k.en) : span_of(p, kv);
      const bool sink = alive && kv < sp.x + p.S;
      const bool alone = alive && sees_one(p, kv, sp.x);
      const int qmax = !alive ? -1 : sink ? sp.y - 1 : min(kv + p.W - 1, sp.y - 1);
      const float up = power2(k.e - P_EXP);
      int qi = k.q_first - 1;  // (group head, query block) pairs, without a division on the way to the scores
      for (int i = 0; i < nloop; ++i, ++n) {
        const uint32_t b = n & 1, slot = n % BWD_STAGES;
        if (++qi == k.q_end) qi = k.q_first;
        const int c0 = qi * 64 + 32 * h;  // query index of column 0 of this half
        const uint32_t bits = span_bits(kv - c0, qmax - c0);
        const Sight sight = sight_of(bits);
        if (!warp_wait(&st_full[b], (n >> 1) & 1, abort_flag, p.err, ERR_WIN_SOFTMAX, p.timeout_ns) ||
            !warp_wait(&qd_full[slot], (n / BWD_STAGES) & 1, abort_flag, p.err, ERR_WIN_SOFTMAX, p.timeout_ns)) {
          ok = false;
          break;
        }
        ptx::tc_fence_after();
        const uint32_t tSb = tmem + 64 * b + lane_base + 32 * h, tdPb = tSb + 128;
        const float4* l2 = reinterpret_cast<const float4*>(sLD + slot * 128 + 32 * h);
        const float4* dd = reinterpret_cast<const float4*>(sLD + slot * 128 + 64 + 32 * h);
        // the query of this key's own row, when it sees nothing else
        const uint32_t own = alone && kv >= c0 && kv < c0 + 32 ? 1u << (kv - c0) : 0u;
        p_ds_step<false>(tSb, tdPb, p.scale_log2, 0.f, 0.f, up, l2, dd, bits, bits & ~own, sight);
        if (total < p.N && qi * 64 + 64 > total) {
          // Q and dO rows behind the last sequence may hold anything: zero them before the dV, dK MMAs
          // multiply them with P = dS = 0 (four panels of 64 rows, 256 threads)
          const int t2 = static_cast<int>(threadIdx.x) - 64, r = t2 & 63;
          if (qi * 64 + r >= total) zero_row128(sQd + slot * 2 * TILE64 + (t2 >> 6) * PANEL64 + r * 128);
          ptx::fence_proxy_async_smem();
        }
        ptx::tmem_st_wait();
        ptx::tc_fence_before();
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(&pds_full[b]);
      }
      if (!ok) break;
      if (nloop > 0) {
        if (!warp_wait(acc_full, blocks & 1, abort_flag, p.err, ERR_WIN_SOFTMAX, p.timeout_ns)) break;
        ++blocks;
        ptx::tc_fence_after();
      }
      // Sink rows that queries beyond the block's reach see: fp32 sums for window_sink_kernel.  A far work's
      // block may hold sinks of other sequences, which its chunk does not see.
      const bool partial = sink && p.nch > 0 && reach64(p, k.kb) * 64 < sp.y && (!k.far || sp.x == k.far_st);
      float* frow = partial ? far_row(p, k.kvh, k.chunk, kv - sp.x) : nullptr;
      uint16_t* drow = p.dQKV + (static_cast<int64_t>(k.shard) * p.N + kv) * p.row_w;
#pragma unroll
      for (int part = 0; part < 2; ++part) {  // dV, dK
        uint32_t r[2][32];
        if (nloop > 0) {
          ptx::tmem_ld32((part ? tdK : tdV) + lane_base + 64 * h, r[0]);
          ptx::tmem_ld32((part ? tdK : tdV) + lane_base + 64 * h + 32, r[1]);
          ptx::tmem_ld_wait();
          if (part == 1) {  // the next block's MMAs may overwrite dV and dK
            ptx::tc_fence_before();
            ptx::mbar_arrive(acc_empty);
          }
        } else {
#pragma unroll
          for (int e = 0; e < 64; ++e) r[e >> 5][e & 31] = 0u;
        }
        const float down = power2(part ? -k.e : -P_EXP);
        if (partial && ok) {
          float* dst = frow + part * HD + 64 * h;
#pragma unroll
          for (int e = 0; e < 64; e += 4) {
            const uint32_t* v = &r[e >> 5][e & 31];
            *reinterpret_cast<float4*>(dst + e) = make_float4(__uint_as_float(v[0]) * down, __uint_as_float(v[1]) * down,
                                                              __uint_as_float(v[2]) * down, __uint_as_float(v[3]) * down);
          }
        } else if (!k.far && ok && kv < p.N) {
          const float mul = part ? p.scale * down : down;
          uint16_t* dst = drow + (part ? k.kcol : k.vcol) + 64 * h;
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            uint32_t v[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              const float x0 = __uint_as_float(r[c >> 1][(c & 1) * 16 + 2 * e]) * mul;
              const float x1 = __uint_as_float(r[c >> 1][(c & 1) * 16 + 2 * e + 1]) * mul;
              v[e] = p.dqkv_f16 ? pack_f16x2(x0, x1) : pack_bf16x2(x0, x1);
            }
            store_16(dst + 16 * c, v, p.wide);
          }
        }
      }
    }
  }

  ptx::tc_fence_before();
  __syncwarp();
  __syncthreads();
  if (warp == 1) {
    __syncwarp();
    ptx::tc_fence_after();
    ptx::tmem_dealloc(tmem, 512);
  }
}

// The larger magnitudes of two pairs of fp16.
__device__ __forceinline__ __half2 max_abs2(__half2 m, uint32_t x) {
  x &= 0x7fff7fffu;
  return __hmax2(m, *reinterpret_cast<const __half2*>(&x));
}

// One 128-query block of a head and the 64-key blocks that it sees.
struct DqWork {
  int shard, jj, qb, kcol, vcol;
  KeyBlocks l;
  int st;  // where the sequence of its rows begins, -1: not one for all rows
  DqWork() = default;
  __device__ DqWork(const WinArgs& p, int w, int total) {
    const int head = w % p.H;
    qb = p.nqb - 1 - w / p.H;
    shard = head / p.hpr;
    jj = head - shard * p.hpr;
    kcol = static_cast<int>(p.kcol0) + (jj / p.Gs) * HD;
    vcol = static_cast<int>(p.vcol0) + (jj / p.Gs) * HD;
    l = key_blocks<6>(p, qb * BQ, total);
    st = common_begin(p, qb * BQ, BQ, total);
  }
  __device__ int count() const { return (l.a1 - l.a0) + (l.b1 - l.b0); }
  __device__ int block(int j) const { return j < l.a1 - l.a0 ? l.a0 + j : l.b0 + j - (l.a1 - l.a0); }
};

__global__ void __launch_bounds__(DQ_THREADS, 1)
    window_dq_kernel(const __grid_constant__ CUtensorMap tm_qkv, const __grid_constant__ CUtensorMap tm_do,
                     const WinArgs p) {
  extern __shared__ uint8_t dsmem[];
  const uint32_t pad = (1024u - (ptx::smem_addr(dsmem) & 1023u)) & 1023u;
  uint8_t* base = dsmem + pad;
  uint8_t* sQ = base;
  uint8_t* sdO = base + TILE;
  uint8_t* sKV = base + 2 * TILE;  // stage s: K_j at s * 2 TILE64, V_j after it
  uint64_t* bars = reinterpret_cast<uint64_t*>(base + 2 * TILE + DQ_STAGES * 2 * TILE64);
  uint64_t* q_full = bars + 0;
  uint64_t* q_empty = bars + 1;                    // the block's last S, dP read Q and dO
  uint64_t* kv_full = bars + 2;                    // [DQ_STAGES]
  uint64_t* kv_empty = bars + 2 + DQ_STAGES;      // [DQ_STAGES]
  uint64_t* s_full = bars + 2 + 2 * DQ_STAGES;    // [2] S, dP of a step in TMEM
  uint64_t* ds_full = bars + 4 + 2 * DQ_STAGES;   // [2] dS written
  uint64_t* acc_full = bars + 6 + 2 * DQ_STAGES;  // [2] dQ of a block complete
  uint64_t* acc_empty = bars + 8 + 2 * DQ_STAGES; // [2] .. and read
  uint64_t* mma_done = bars + 10 + 2 * DQ_STAGES;
  uint64_t* d_full = bars + 11 + 2 * DQ_STAGES;   // [2] D of a block
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 13 + 2 * DQ_STAGES);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  WorkQueue<DqWork, 13> queue(reinterpret_cast<uint8_t*>(bars) + 256);
  volatile float* sD =  // of two blocks in turn, 2^e D [128] of the rows, then 2^e [4] of each 32
      reinterpret_cast<volatile float*>(reinterpret_cast<uint8_t*>(bars) + 256 + QUEUE_SMEM);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    ptx::mbar_init(q_full, 1);
    ptx::mbar_init(q_empty, 1);
    for (int s = 0; s < DQ_STAGES; ++s) {
      ptx::mbar_init(&kv_full[s], 1);
      ptx::mbar_init(&kv_empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      ptx::mbar_init(&s_full[b], 1);
      ptx::mbar_init(&ds_full[b], 8);
      ptx::mbar_init(&acc_full[b], 1);
      ptx::mbar_init(&acc_empty[b], 4);
      ptx::mbar_init(&d_full[b], 4);
    }
    ptx::mbar_init(mma_done, 1);
    queue.init();
    *abort_flag = 0;
    ptx::fence_mbar_init();
  }
  if (warp == 1) {
    ptx::tmem_alloc(tmem_slot, 512);
    ptx::tmem_relinquish();
  }
  ptx::tc_fence_before();
  __syncwarp();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  ptx::griddep_wait();
  ptx::griddep_launch_dependents();
  const int total = total_rows(p);
  // TMEM columns: S_0 | S_1 (64 each) | dP_0 | dP_1 (64 each) | dQ of this block and of the one before (128 each).

  if (warp == 0) {
    if (lane == 0) {
      ptx::tma_prefetch_desc(&tm_qkv);
      ptx::tma_prefetch_desc(&tm_do);
      uint32_t issued = 0, blocks = 0;
      bool ok = true;
      for (int w = blockIdx.x; ok && w >= 0; w = queue.next(abort_flag, p.err, ERR_WIN_PRODUCER, p.timeout_ns)) {
        const DqWork k(p, w, total);
        const int nkv = k.count();
        ok = queue.post(k, abort_flag, p.err, ERR_WIN_PRODUCER, p.timeout_ns);
        if (!ok) break;
        if (nkv == 0) continue;
        ok = blocks == 0 ||
             ptx::mbar_wait(q_empty, (blocks - 1) & 1, abort_flag, p.err, ERR_WIN_PRODUCER, p.timeout_ns);
        if (!ok) break;
        ptx::mbar_arrive_expect_tx(q_full, 2 * TILE);
        ++blocks;
        tma_tile128(sQ, &tm_qkv, q_full, k.jj * HD, k.qb * BQ, k.shard);
        tma_tile128(sdO, &tm_do, q_full, k.jj * HD, k.qb * BQ, k.shard);
        for (int j = 0; j < nkv; ++j, ++issued) {
          if (j + DQ_AHEAD >= nkv) queue.ask();
          const uint32_t slot = issued % DQ_STAGES;
          if (!ptx::mbar_wait(&kv_empty[slot], ((issued / DQ_STAGES) & 1) ^ 1u, abort_flag, p.err, ERR_WIN_PRODUCER,
                              p.timeout_ns)) {
            ok = false;
            break;
          }
          uint8_t* dst = sKV + slot * 2 * TILE64;
          ptx::mbar_arrive_expect_tx(&kv_full[slot], 2 * TILE64);
          tma_tile64(dst, &tm_qkv, &kv_full[slot], k.kcol, k.block(j) * 64, k.shard);
          tma_tile64(dst + TILE64, &tm_qkv, &kv_full[slot], k.vcol, k.block(j) * 64, k.shard);
        }
      }
      if (ok) queue.post_end(abort_flag, p.err, ERR_WIN_PRODUCER, p.timeout_ns);
      queue.drain(p.err, ERR_WIN_DRAIN, p.timeout_ns);
      volatile int never = 0;
      if (blocks > 0) ptx::mbar_wait(q_full, (blocks - 1) & 1, &never, p.err, ERR_WIN_DRAIN, p.timeout_ns);
      for (uint32_t j = (issued > DQ_STAGES ? issued - DQ_STAGES : 0); j < issued; ++j)
        ptx::mbar_wait(&kv_full[j % DQ_STAGES], (j / DQ_STAGES) & 1, &never, p.err, ERR_WIN_DRAIN, p.timeout_ns);
    }
  } else if (warp == 1) {
    if (ptx::elect_one()) {
      constexpr uint32_t idesc_s = ptx::idesc_f16_f32(128, 64, false, false);  // S, dP
      constexpr uint32_t idesc_q = ptx::idesc_f16_f32(128, 128, false, true);  // dQ = dS K
      // Descriptors are formed once; a tile or a k-step is an addition.
      const uint64_t dQ = ptx::sdesc_sw128(ptx::smem_addr(sQ), 16, 1024);
      const uint64_t ddO = ptx::sdesc_sw128(ptx::smem_addr(sdO), 16, 1024);
      const uint64_t dKV = ptx::sdesc_sw128(ptx::smem_addr(sKV), 16, 1024);         // rows as they are
      const uint64_t dKVT = ptx::sdesc_sw128(ptx::smem_addr(sKV), PANEL64, 1024);   // .. transposed
      auto issue_s = [&](uint32_t n) {
        const uint32_t slot = n % DQ_STAGES, b = n & 1;
        if (!ptx::mbar_wait(&kv_full[slot], (n / DQ_STAGES) & 1, abort_flag, p.err, ERR_WIN_MMA, p.timeout_ns))
          return false;
        ptx::tc_fence_after();
        const uint64_t kv = ptx::sdesc_at(dKV, slot * 2 * TILE64);
#pragma unroll
        for (int kk = 0; kk < 8; ++kk)
          ptx::mma_bf16(tmem + 64 * b, ptx::sdesc_at(dQ, kstep(kk, PANEL)), ptx::sdesc_at(kv, kstep(kk, PANEL64)), idesc_s,
                        kk > 0 ? 1u : 0u);
#pragma unroll
        for (int kk = 0; kk < 8; ++kk)
          ptx::mma_bf16(tmem + 128 + 64 * b, ptx::sdesc_at(ddO, kstep(kk, PANEL)),
                        ptx::sdesc_at(kv, TILE64 + kstep(kk, PANEL64)), idesc_s, kk > 0 ? 1u : 0u);
        ptx::mma_commit(&s_full[b]);
        return true;
      };
      uint32_t n = 0, blocks = 0;
      bool ok = true;
      DqWork k;
      while (ok && queue.read<false>(k, abort_flag, p.err, ERR_WIN_MMA, p.timeout_ns)) {
        const int nkv = k.count();
        if (nkv == 0) continue;
        ok = ptx::mbar_wait(q_full, blocks & 1, abort_flag, p.err, ERR_WIN_MMA, p.timeout_ns) && issue_s(n);
        if (ok && nkv == 1) ptx::mma_commit(q_empty);
        for (int j = 0; ok && j < nkv; ++j, ++n) {
          if (j + 1 < nkv) {
            if (!issue_s(n + 1)) {
              ok = false;
              break;
            }
            if (j + 2 == nkv) ptx::mma_commit(q_empty);
          }
          const uint32_t b = n & 1, slot = n % DQ_STAGES;
          if (!ptx::mbar_wait(&ds_full[b], (n >> 1) & 1, abort_flag, p.err, ERR_WIN_MMA, p.timeout_ns) ||
              (j == 0 && blocks > 1 &&
               !ptx::mbar_wait(&acc_empty[blocks & 1], ((blocks >> 1) - 1) & 1, abort_flag, p.err, ERR_WIN_MMA,
                               p.timeout_ns))) {
            ok = false;
            break;
          }
          ptx::tc_fence_after();
          const uint64_t kv = ptx::sdesc_at(dKVT, slot * 2 * TILE64);
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            ptx::mma_f16_ts(tmem + 256 + 128 * (blocks & 1), tmem + 64 * b + half_split_col(kk),
                            ptx::sdesc_at(kv, kk * 2048), idesc_q, (j > 0 || kk > 0) ? 1u : 0u);
          ptx::mma_commit(&kv_empty[slot]);
        }
        if (!ok) break;
        ptx::mma_commit(&acc_full[blocks & 1]);
        ++blocks;
      }
      ptx::mma_commit(mma_done);
      volatile int never = 0;
      ptx::mbar_wait(mma_done, 0, &never, p.err, ERR_WIN_DRAIN, p.timeout_ns);
    }
  } else if (warp < 10) {
    // Compute warps: lane quarter warp & 3 (query rows), column half h of each 64-key block.
    const int quad = warp & 3, h = (warp - 2) >> 2;
    const uint32_t lane_base = static_cast<uint32_t>(quad * 32) << 16;
    uint32_t n = 0, blocks = 0;
    bool ok = true;
    DqWork k;
    while (ok && queue.read<true>(k, abort_flag, p.err, ERR_WIN_SOFTMAX, p.timeout_ns)) {
      const int nkv = k.count();
      const int q = k.qb * BQ + quad * 32 + lane;
      const int64_t vec = (static_cast<int64_t>(k.shard) * p.hpr + k.jj) * p.N;
      const bool alive = q < total;
      const float nl = alive ? -(p.lse[vec + q] * kLog2e) : 0.0f;
      float nd = 0.0f, up = 1.0f;
      if (nkv > 0) {
        ok = warp_wait(&d_full[blocks & 1], (blocks >> 1) & 1, abort_flag, p.err, ERR_WIN_SOFTMAX, p.timeout_ns);
        if (!ok) break;
        nd = -sD[(blocks & 1) * 132 + quad * 32 + lane];
        up = sD[(blocks & 1) * 132 + 128 + quad];
      }
      const int st = !alive ? 0 : k.st >= 0 ? k.st : span_of(p, q).x;
      const bool sees = alive && !sees_one(p, q, st);
      const int wlo = sees ? max(st, q - p.W + 1) : 1, whi = sees ? q : 0;  // visible window keys
      const int shi = sees && p.S > 0 ? min(st + p.S - 1, q) : -1;          // visible sinks st .. shi
      for (int j = 0; j < nkv; ++j, ++n) {
        const uint32_t b = n & 1;
        const int k0 = k.block(j) * 64, c0 = k0 + 32 * h;
        const uint32_t bits = span_bits(wlo - c0, whi - c0) | span_bits(st - c0, shi - c0);
        const Sight sight = sight_of(bits);
        if (!warp_wait(&s_full[b], (n >> 1) & 1, abort_flag, p.err, ERR_WIN_SOFTMAX, p.timeout_ns)) {
          ok = false;
          break;
        }
        ptx::tc_fence_after();
        const uint32_t tSb = tmem + 64 * b + lane_base + 32 * h, tdPb = tSb + 128;
        p_ds_step<true>(tSb, tdPb, p.scale_log2, nl, nd, up, nullptr, nullptr, bits, bits, sight);
        if (total < p.N && k0 + 64 > total) {
          // K rows behind the last sequence may hold anything: zero them before the dQ MMA multiplies
          // them with dS = 0 (two panels of 64 rows)
          const int slot = static_cast<int>(n % DQ_STAGES), t2 = static_cast<int>(threadIdx.x) - 64, r = t2 & 63;
          ok = warp_wait(&kv_full[slot], (n / DQ_STAGES) & 1, abort_flag, p.err, ERR_WIN_SOFTMAX, p.timeout_ns) && ok;
          if (t2 < 128 && k0 + r >= total) zero_row128(sKV + slot * 2 * TILE64 + (t2 >> 6) * PANEL64 + r * 128);
          ptx::fence_proxy_async_smem();
        }
        ptx::tmem_st_wait();
        ptx::tc_fence_before();
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(&ds_full[b]);
      }
      if (!ok) break;
      if (nkv > 0) ++blocks;
    }
  } else {
    // Output warps: D, and the e of dS, of a block before the compute warps come to it, dQ of the one before while
    // they are at it; a row a thread.  (D = rowsum(dO O) as a kernel of its own took 83 us at N 16384, 64 heads; by the compute
    // warps from an O tile beside Q and dO it was 2,400 of 27,000 cycles of a block: 656 us for the kernel, not 632.)
    const int quad = warp & 3, row = quad * 32 + lane;
    const uint32_t lane_base = static_cast<uint32_t>(quad * 32) << 16;
    auto form_d = [&](const DqWork& k, uint32_t block) {  // returns 2^-e of this warp's rows
      // the largest sum|v| of the key blocks that the tile sees, the first 32 of them beside dO and O
      const int a0 = k.l.a0 >> 1, na = k.l.a1 > k.l.a0 ? ((k.l.a1 + 1) >> 1) - a0 : 0, b0 = k.l.b0 >> 1;
      const int nv = na + ((k.l.b1 + 1) >> 1) - b0;
      auto v_at = [&](int i) {
        return i < nv ? *value_bound(p, k.shard, k.vcol, i < na ? a0 + i : b0 + i - na) : 0.0f;
      };
      float vm = v_at(lane);
      __half2 top = __float2half2_rn(0.0f);  // max|dO| of the rows
      // half a warp a row, 16 rows in flight
      const int half = lane >> 4;
      const int64_t at =
          (static_cast<int64_t>(k.shard) * p.N + k.qb * BQ + quad * 32) * p.dt + k.jj * HD + 8 * (lane & 15);
      const int rows = min(32, total - (k.qb * BQ + quad * 32));  // of this warp's in a sequence
      float D = 0.0f;
#pragma unroll 1
      for (int r0 = 0; r0 < rows; r0 += 16) {
        uint4 o[8], g[8];
#pragma unroll
        for (int u = 0; u < 8; ++u) {
          const int64_t off = at + min(r0 + 2 * u + half, rows - 1) * p.dt;
          o[u] = *reinterpret_cast<const uint4*>(p.O + off);
          g[u] = *reinterpret_cast<const uint4*>(p.dO + off);
        }
#pragma unroll
        for (int u = 0; u < 8; ++u) {
          const uint32_t ow[4] = {o[u].x, o[u].y, o[u].z, o[u].w}, gw[4] = {g[u].x, g[u].y, g[u].z, g[u].w};
          float sum = 0.0f;
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            float o0, o1, g0, g1;
            unpack_bf16x2(ow[e], o0, o1);
            unpack_f16x2(gw[e], g0, g1);
            sum = fmaf(g0, o0, fmaf(g1, o1, sum));
            top = max_abs2(top, gw[e]);
          }
#pragma unroll
          for (int m = 8; m > 0; m >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, m);
          const float even = __shfl_sync(0xffffffffu, sum, 0), odd = __shfl_sync(0xffffffffu, sum, 16);
          if (lane < rows && (lane & ~1) == r0 + 2 * u) D = lane & 1 ? odd : even;
        }
      }
#pragma unroll 4
      for (int i = lane + 32; i < nv; i += 32) vm = fmaxf(vm, v_at(i));
      auto warp_max = [](float x) {  // of values that are not negative
        return __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(x)));
      };
      const float bound = warp_max(__half2float(__hmax(__low2half(top), __high2half(top)))) * warp_max(vm);
      const int e = ds_exponent(bound);
      const float up = power2(e);
      sD[(block & 1) * 132 + row] = D * up;  // 0 for the rows behind the last sequence
      if (lane == 0) sD[(block & 1) * 132 + 128 + quad] = up;
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(&d_full[block & 1]);
      // for dK, dV
      const int64_t vec = (static_cast<int64_t>(k.shard) * p.hpr + k.jj) * p.N;
      if (lane < rows && k.qb * BQ + row > 0) p.Dvec[vec + k.qb * BQ + row] = D;
      if (lane == 0) atomicMax(row_bound(p, k.shard, k.jj), __float_as_uint(bound));  // a maximum: the order does not matter
      return power2(-e);
    };
    auto row_of = [&](const DqWork& k) {
      return p.dQKV + (static_cast<int64_t>(k.shard) * p.N + k.qb * BQ + row) * p.row_w + k.jj * HD;
    };
    uint32_t blocks = 0;  // whose D is formed
    DqWork k;
    uint16_t* out = nullptr;  // this thread's row of the block whose dQ is to be stored
    float mul = 0.0f, mul_new = 0.0f;  // .. and its factor, scale 2^-e, and that of the block being formed
    bool stores = false, more = true;
    while (more) {
      more = queue.read<true>(k, abort_flag, p.err, ERR_WIN_SOFTMAX, p.timeout_ns);
      const bool work = more && k.count() > 0;
      if (work) mul_new = p.scale * form_d(k, blocks);
      if (stores && (work || !more)) {
        const uint32_t done = blocks - 1, pb = done & 1;
        if (!warp_wait(&acc_full[pb], (done >> 1) & 1, abort_flag, p.err, ERR_WIN_SOFTMAX, p.timeout_ns)) break;
        ptx::tc_fence_after();
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          uint32_t r[32];
          ptx::tmem_ld32(tmem + 256 + 128 * pb + lane_base + 32 * c, r);
          ptx::tmem_ld_wait();
          if (c == 3) {
            ptx::tc_fence_before();
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(&acc_empty[pb]);
          }
          if (out) {
#pragma unroll
            for (int u = 0; u < 2; ++u) {
              uint32_t v[8];
#pragma unroll
              for (int e = 0; e < 8; ++e) {
                const float x0 = __uint_as_float(r[16 * u + 2 * e]) * mul;
                const float x1 = __uint_as_float(r[16 * u + 2 * e + 1]) * mul;
                v[e] = p.dqkv_f16 ? pack_f16x2(x0, x1) : pack_bf16x2(x0, x1);
              }
              store_16(out + 32 * c + 16 * u, v, p.wide);
            }
          }
        }
      }
      if (!more) break;
      if (work) {
        out = k.qb * BQ + row < p.N ? row_of(k) : nullptr;
        mul = mul_new;
        stores = true;
        ++blocks;
      } else if (k.qb * BQ + row < p.N) {  // a block behind the last sequence
        zero_row128(reinterpret_cast<uint8_t*>(row_of(k)));
        zero_row128(reinterpret_cast<uint8_t*>(row_of(k) + 64));
      }
    }
  }

  ptx::tc_fence_before();
  __syncwarp();
  __syncthreads();
  if (warp == 1) {
    __syncwarp();
    ptx::tc_fence_after();
    ptx::tmem_dealloc(tmem, 512);
  }
}

// dV, dK of the sink rows that queries beyond their block's reach see: the block's own sums, then the
// chunks' in order.  One CTA per (KV head, 128 rows); its warps take dV and dK of the rows found in turn,
// a lane has 4 columns, the loads of 8 chunks are in flight together.
constexpr int SINK_THREADS = 512;
__global__ void __launch_bounds__(SINK_THREADS) window_sink_kernel(const WinArgs p) {
  __shared__ int rows[BKV];
  __shared__ int found[4];
  ptx::griddep_wait();
  ptx::griddep_launch_dependents();
  const int kvh = blockIdx.x % p.Hkv, kb = static_cast<int>(blockIdx.x / p.Hkv);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int far0 = reach64(p, kb) * 64;
  const int total = total_rows(p);
  bool mine = false;
  const int r = kb * BKV + static_cast<int>(threadIdx.x);
  uint32_t hits = 0;
  if (warp < 4) {
    const int2 sp = r < total ? span_of(p, r) : make_int2(0, 0);
    mine = r < total && r < sp.x + p.S && far0 < sp.y;
    hits = __ballot_sync(0xffffffffu, mine);
    if (lane == 0) found[warp] = __popc(hits);
  }
  __syncthreads();
  int before = 0;
  for (int w = 0; w < warp && w < 4; ++w) before += found[w];
  if (mine) rows[before + __popc(hits & ((1u << lane) - 1))] = r;
  const int count = found[0] + found[1] + found[2] + found[3];
  __syncthreads();
  const int shard = kvh / p.kv_t, jl = kvh - shard * p.kv_t;
  for (int i = warp; i < 2 * count; i += SINK_THREADS / 32) {  // dV, dK of each row
    const int kv = rows[i >> 1], part = i & 1;
    const int2 sp = span_of(p, kv);
    const int c_lo = far0 / p.C, c_hi = (sp.y - 1) / p.C;
    auto load = [&](int c) {
      return __ldcg(reinterpret_cast<const float4*>(far_row(p, kvh, c, kv - sp.x) + part * HD) + lane);
    };
    float4 sum = load(p.nch + c_lo);
    for (int c = c_lo; c <= c_hi; c += 8) {
      float4 v[8];
#pragma unroll
      for (int u = 0; u < 8; ++u) v[u] = c + u <= c_hi ? load(c + u) : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        sum.x += v[u].x;
        sum.y += v[u].y;
        sum.z += v[u].z;
        sum.w += v[u].w;
      }
    }
    const float mul = part ? p.scale : 1.0f;
    auto two = [&](float x, float y) { return p.dqkv_f16 ? pack_f16x2(x * mul, y * mul) : pack_bf16x2(x * mul, y * mul); };
    uint16_t* drow = p.dQKV + (static_cast<int64_t>(shard) * p.N + kv) * p.row_w + (part ? p.kcol0 : p.vcol0) + jl * HD;
    *reinterpret_cast<uint2*>(drow + 4 * lane) = make_uint2(two(sum.x, sum.y), two(sum.z, sum.w));
  }
}

// --------------------------------------------------------------- sequences
// span[r] = the (begin, end) of row r's sequence, from the n + 1 boundaries in cu; end = r: none
// (behind the last).  Boundaries that are out of order or out of range are reported, and clamped
// so that every span holds its row and stays in [0, N).  Called by `threads` >= N threads, i = 0, 1, ..
__device__ __forceinline__ void write_spans(const int32_t* cu, int n, int N, int* total_out, int2* span, int* err,
                                            int64_t i, int64_t threads) {
  const int total = max(0, min(cu[n], N));
  if (i == 0) {
    *total_out = total;
    if (cu[0] != 0 || cu[n] > N) atomicCAS(err, 0, kErrSeqlens);
  }
  for (int64_t k = i; k < n; k += threads)
    if (cu[k] > cu[k + 1]) atomicCAS(err, 0, kErrSeqlens);
  if (i >= N) return;
  const int r = static_cast<int>(i);
  if (r >= total) {
    span[r] = make_int2(r, r);
    return;
  }
  int lo = 0, hi = n - 1;  // the last sequence that begins at or before r
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (cu[mid] <= r) lo = mid;
    else hi = mid - 1;
  }
  span[r] = make_int2(max(0, min(cu[lo], r)), min(max(cu[lo + 1], r + 1), total));
}

__global__ void __launch_bounds__(256) window_spans_kernel(const int32_t* cu, int n, int N, int* total_out, int2* span,
                                                           int* err) {
  ptx::griddep_wait();
  ptx::griddep_launch_dependents();
  write_spans(cu, n, N, total_out, span, err, static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x,
              static_cast<int64_t>(gridDim.x) * blockDim.x);
}

// Before the backward: the spans (when there are boundaries), and per (KV head, 128-key block) the largest sum|v|
// of its rows that belong to a sequence, for the powers of two of dS (see the top); row_bound() starts at 0.
// One CTA a block: half a warp a row, the loads of a warp's 16 rows in flight together.  V is read once, HBM-bound.
constexpr int PREP_THREADS = 256;
__global__ void __launch_bounds__(PREP_THREADS) window_prep_kernel(const WinArgs p, const int32_t* cu, int n_seq,
                                                                   int* total_out, int2* span) {
  __shared__ float warp_top[PREP_THREADS / 32];
  ptx::griddep_wait();
  ptx::griddep_launch_dependents();
  const int kvh = blockIdx.x % p.Hkv, kb = static_cast<int>(blockIdx.x / p.Hkv);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int shard = kvh / p.kv_t, jl = kvh - shard * p.kv_t;
  const int total = cu ? max(0, min(cu[n_seq], p.N)) : p.N;
  const int r0 = kb * BKV + warp * 16 + (lane >> 4);
  const uint16_t* v = p.QKV + static_cast<int64_t>(shard) * p.N * p.row_w + p.vcol0 + jl * HD + 8 * (lane & 15);
  uint4 w[8];
#pragma unroll
  for (int u = 0; u < 8; ++u)
    w[u] = r0 + 2 * u < total ? *reinterpret_cast<const uint4*>(v + (r0 + 2 * u) * p.row_w) : make_uint4(0u, 0u, 0u, 0u);
  if (cu && kvh == 0 && threadIdx.x < BKV)
    write_spans(cu, n_seq, p.N, total_out, span, p.err, static_cast<int64_t>(kb) * BKV + threadIdx.x,
                static_cast<int64_t>(p.nqb) * BKV);
  if (kb == 0 && threadIdx.x == 0) *row_bound(p, shard, jl * p.Gs) = 0u;
  float top = 0.0f;
#pragma unroll
  for (int u = 0; u < 8; ++u) {
    const uint32_t x[4] = {w[u].x, w[u].y, w[u].z, w[u].w};
    float sum = 0.0f;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      float v0, v1;
      unpack_f16x2(x[e], v0, v1);
      sum += fabsf(v0) + fabsf(v1);
    }
#pragma unroll
    for (int m = 8; m > 0; m >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, m);
    top = fmaxf(top, sum);
  }
  top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 16));
  if (lane == 0) warp_top[warp] = top;
  __syncthreads();
  if (threadIdx.x == 0) {
#pragma unroll
    for (int k = 0; k < PREP_THREADS / 32; ++k) top = fmaxf(top, warp_top[k]);
    *value_bound(p, shard, static_cast<int>(p.vcol0) + jl * HD, kb) = top;
  }
}

inline size_t up256(size_t x) { return (x + 255) & ~static_cast<size_t>(255); }

// Workspace: [total, padded to 256 bytes][span of every row] when there are sequences, then `far`.
size_t span_bytes(int64_t N, int64_t n_seq) { return n_seq > 0 ? 256 + up256(static_cast<size_t>(N) * sizeof(int2)) : 0; }

struct FarPlan {
  int C = 0, nch = 0, nsb = 0;
  size_t bytes = 0;
};
// Chunk rows: at most the window (see the top), or one 128-row block under a narrow one; 2048 keeps a
// far CTA's loop no longer than that of a key block at W = 1920.
FarPlan far_plan(int64_t N, int Hkv, int64_t W, int64_t S, int64_t n_seq) {
  FarPlan f;
  if (S < 1 || N < W + BKV) return f;
  f.C = W >= 256 ? static_cast<int>((W < 2048 ? W : 2048) / BKV * BKV) : BKV;
  f.nch = static_cast<int>((N + f.C - 1) / f.C);
  f.nsb = static_cast<int>(n_seq > 0 ? (S + BKV - 2) / BKV + 1 : (S + BKV - 1) / BKV);
  f.bytes = static_cast<size_t>(Hkv) * 2 * f.nch * S * 2 * HD * sizeof(float);
  return f;
}

// Window and sinks as they act on N rows: neither reaches further, and where they leave no key of N hidden
// (a hidden key is W back and S from the first) the attention is the full causal one: no sinks then, so
// no far works and no room for them, however many sinks were asked for.
struct Reach {
  int64_t W, S;
};
Reach reach_of(int64_t N, int64_t window, int64_t n_sink) {
  const Reach r{window < N ? window : N, n_sink < N ? n_sink : N};
  return r.W + r.S >= N ? Reach{N, 0} : r;
}

tp_status check_window(int64_t N, int64_t d, int n_heads, int n_kv, int head_dim, int t, const WindowAttn& o,
                       AttnShape& sh) {
  if (N < 0 || d < 1 || n_heads < 1 || n_kv < 1 || t < 1 || head_dim < 1) return TP_ERR_INVALID_ARG;
  if (o.window < 1 || o.n_sink < 0 || o.n_seq < 0 || (o.n_seq > 0) != (o.cu_seqlens != nullptr))
    return TP_ERR_INVALID_ARG;
  if (!attn_shape(d, n_heads, n_kv, head_dim, t, sh)) return TP_ERR_SHAPE;
  // row indices and their sums with the window fit 32 bits (2^29 rows of QKV have 400 GB)
  if (N > (1LL << 29) || o.n_seq > (1LL << 30)) return TP_ERR_SHAPE;
  if (!aligned4(o.cu_seqlens)) return TP_ERR_ALIGN;
  return TP_OK;
}

// Pairs of query tiles of the forward, and works of the two backward kernels.
int64_t fwd_works(int64_t N, int n_heads, const AttnShape& sh) {
  const int64_t nqb = (N + BQ - 1) / BQ;
  return sh.Gs % 2 == 0 ? n_heads / 2 * nqb : n_heads * ((nqb + 1) / 2);
}
struct BwdWorks {
  int64_t q, kv, far;
};
BwdWorks bwd_works(int64_t N, int n_heads, int Hkv, const FarPlan& f) {
  const int64_t nqb = (N + BQ - 1) / BQ;
  return BwdWorks{n_heads * nqb, Hkv * nqb, static_cast<int64_t>(Hkv) * f.nch * f.nsb};
}

void fill_args(WinArgs& a, int64_t N, int n_heads, int t, const WindowAttn& o, const AttnShape& sh, float scale) {
  a.N = static_cast<int>(N);
  a.H = n_heads;
  a.hpr = n_heads / t;
  a.Gs = sh.Gs;
  a.kv_t = sh.kv_t;
  a.Hkv = t * sh.kv_t;
  const Reach r = reach_of(N, o.window, o.n_sink);
  a.W = static_cast<int>(r.W);
  a.S = static_cast<int>(r.S);
  a.by_head = sh.Gs % 2 == 0;
  a.nqb = static_cast<int>((N + BQ - 1) / BQ);
  a.dt = sh.dt;
  a.row_w = sh.row_w;
  a.kcol0 = sh.kcol0;
  a.vcol0 = sh.vcol0;
  a.scale = scale;
  a.scale_log2 = scale * kLog2e;
  a.timeout_ns = wait_timeout_ns();
}

// The spans of cu_seqlens' rows into the head of the workspace.
tp_status make_spans(WinArgs& a, const WindowAttn& o, void* ws, cudaStream_t s) {
  if (o.n_seq < 1) return TP_OK;
  int* total = static_cast<int*>(ws);
  int2* span = reinterpret_cast<int2*>(static_cast<uint8_t*>(ws) + 256);
  TP_CUDA_CHECK(launch_pdl(window_spans_kernel, dim3(static_cast<unsigned>((a.N + 255) / 256)), dim3(256), 0, s,
                           o.cu_seqlens, static_cast<int>(o.n_seq), a.N, total, span, a.err));
  count_launch();
  a.total = total;
  a.span = span;
  return TP_OK;
}

}  // namespace

size_t window_attn_fwd_ws_bytes(int64_t N, int64_t n_seq) { return N < 0 || n_seq < 0 ? 0 : span_bytes(N, n_seq); }

tp_status window_attn_fwd_ok(const uint16_t* QKV, int64_t N, int64_t d, int n_heads, int n_kv, int head_dim, int t,
                             const WindowAttn& o, const uint16_t* O, const float* lse, const void* ws, size_t ws_bytes) {
  AttnShape sh;
  TP_RETURN_IF(check_window(N, d, n_heads, n_kv, head_dim, t, o, sh));
  if (N == 0) return TP_OK;
  if (!QKV || !O || !lse) return TP_ERR_INVALID_ARG;
  if (!aligned16(QKV) || !aligned16(O) || !aligned4(lse)) return TP_ERR_ALIGN;
  const size_t qkv_bytes = static_cast<size_t>(t) * N * sh.row_w * 2, o_bytes = static_cast<size_t>(t) * N * sh.dt * 2;
  const size_t lse_bytes = static_cast<size_t>(n_heads) * N * 4;
  if (overlap(QKV, qkv_bytes, O, o_bytes) || overlap(QKV, qkv_bytes, lse, lse_bytes) ||
      overlap(O, o_bytes, lse, lse_bytes))
    return TP_ERR_INVALID_ARG;
  if (o.n_seq > 0) {
    if (!ws || ws_bytes < span_bytes(N, o.n_seq)) return TP_ERR_WORKSPACE;
    if ((reinterpret_cast<uintptr_t>(ws) & 255u) != 0) return TP_ERR_ALIGN;
  }
  return fwd_works(N, n_heads, sh) > INT_MAX ? TP_ERR_SHAPE : TP_OK;
}

tp_status run_window_attn_fwd(const uint16_t* QKV, int64_t N, int64_t d, int n_heads, int n_kv, int head_dim, int t,
                              const WindowAttn& o, float scale, uint16_t* O, float* lse, int zero_pad, void* ws,
                              size_t ws_bytes, cudaStream_t s) {
  TP_RETURN_IF(window_attn_fwd_ok(QKV, N, d, n_heads, n_kv, head_dim, t, o, O, lse, ws, ws_bytes));
  if (N == 0) return TP_OK;
  AttnShape sh;
  TP_RETURN_IF(check_window(N, d, n_heads, n_kv, head_dim, t, o, sh));
  WinArgs a{};
  fill_args(a, N, n_heads, t, o, sh, scale);
  const int64_t grid = fwd_works(N, n_heads, sh);
  TP_RETURN_IF(ready());
  a.err = device_error_word();
  a.QKV = QKV;
  a.O = O;
  a.lse = lse;
  a.wide = (reinterpret_cast<uintptr_t>(O) & 31u) == 0;
  a.zero_pad = zero_pad;
  CUtensorMap map;
  if (!make_map_3d_bf16(&map, QKV, sh.row_w, N, t, sh.row_w * 2, N * sh.row_w * 2, 64, 128))
    return TP_FAIL_DETAIL("cuTensorMapEncodeTiled failed for QKV");
  static bool configured[64] = {};
  int dev = 0;
  TP_CUDA_CHECK(cudaGetDevice(&dev));
  if (dev < 0 || dev >= 64) return TP_ERR_CUDA;
  if (!configured[dev]) {
    TP_CUDA_CHECK(cudaFuncSetAttribute(window_fwd_kernel<false>, cudaFuncAttributeMaxDynamicSharedMemorySize, FWD_SMEM));
    TP_CUDA_CHECK(cudaFuncSetAttribute(window_fwd_kernel<true>, cudaFuncAttributeMaxDynamicSharedMemorySize, FWD_SMEM));
    configured[dev] = true;
  }
  TP_RETURN_IF(make_spans(a, o, ws, s));
  auto kernel = !(a.scale_log2 >= FLT_MIN) ? window_fwd_kernel<true> : window_fwd_kernel<false>;
  TP_CUDA_CHECK(launch_pdl(kernel, dim3(static_cast<unsigned>(grid)), dim3(FWD_THREADS), FWD_SMEM, s, map, a));
  count_launch();
  return TP_OK;
}

size_t window_attn_bwd_ws_bytes(int64_t N, int64_t d, int n_heads, int n_kv, int head_dim, int t, int64_t window,
                                int64_t n_sink, int64_t n_seq) {
  AttnShape sh;
  if (N < 0 || window < 1 || n_sink < 0 || n_seq < 0 || !attn_shape(d, n_heads, n_kv, head_dim, t, sh)) return 0;
  const Reach r = reach_of(N, window, n_sink);
  return span_bytes(N, n_seq) + far_plan(N, t * sh.kv_t, r.W, r.S, n_seq).bytes;
}

tp_status window_attn_bwd_ok(const uint16_t* QKV, const uint16_t* O, const uint16_t* dO, const float* lse, int64_t N,
                             int64_t d, int n_heads, int n_kv, int head_dim, int t, const WindowAttn& o,
                             const float* Dvec, const uint16_t* dQKV, const void* ws, size_t ws_bytes) {
  AttnShape sh;
  TP_RETURN_IF(check_window(N, d, n_heads, n_kv, head_dim, t, o, sh));
  if (N == 0) return TP_OK;
  if (!QKV || !O || !dO || !lse || !Dvec || !dQKV) return TP_ERR_INVALID_ARG;
  if (!aligned16(QKV) || !aligned16(O) || !aligned16(dO) || !aligned16(dQKV) || !aligned4(lse) || !aligned4(Dvec))
    return TP_ERR_ALIGN;
  const size_t qkv_bytes = static_cast<size_t>(t) * N * sh.row_w * 2, o_bytes = static_cast<size_t>(t) * N * sh.dt * 2;
  const size_t lse_bytes = static_cast<size_t>(n_heads) * N * 4;
  auto meets_input = [&](const void* p, size_t bytes) {
    return overlap(p, bytes, QKV, qkv_bytes) || overlap(p, bytes, O, o_bytes) || overlap(p, bytes, dO, o_bytes) ||
           overlap(p, bytes, lse, lse_bytes);
  };
  if (meets_input(dQKV, qkv_bytes) || meets_input(Dvec, lse_bytes) || overlap(dQKV, qkv_bytes, Dvec, lse_bytes))
    return TP_ERR_INVALID_ARG;
  const size_t need = window_attn_bwd_ws_bytes(N, d, n_heads, n_kv, head_dim, t, o.window, o.n_sink, o.n_seq);
  if (need > 0 && (!ws || ws_bytes < need)) return TP_ERR_WORKSPACE;
  if (need > 0 && (reinterpret_cast<uintptr_t>(ws) & 255u) != 0) return TP_ERR_ALIGN;
  const Reach r = reach_of(N, o.window, o.n_sink);
  const BwdWorks w = bwd_works(N, n_heads, t * sh.kv_t, far_plan(N, t * sh.kv_t, r.W, r.S, o.n_seq));
  return w.q > INT_MAX || w.far + w.kv > INT_MAX ? TP_ERR_SHAPE : TP_OK;
}

tp_status run_window_attn_bwd(const uint16_t* QKV, const uint16_t* O, const uint16_t* dO, const float* lse, int64_t N,
                              int64_t d, int n_heads, int n_kv, int head_dim, int t, const WindowAttn& o, float scale,
                              float* Dvec, uint16_t* dQKV, int dqkv_f16, void* ws, size_t ws_bytes, cudaStream_t s) {
  TP_RETURN_IF(window_attn_bwd_ok(QKV, O, dO, lse, N, d, n_heads, n_kv, head_dim, t, o, Dvec, dQKV, ws, ws_bytes));
  if (N == 0) return TP_OK;
  AttnShape sh;
  TP_RETURN_IF(check_window(N, d, n_heads, n_kv, head_dim, t, o, sh));
  WinArgs a{};
  fill_args(a, N, n_heads, t, o, sh, scale);
  const FarPlan f = far_plan(N, a.Hkv, a.W, a.S, o.n_seq);
  const BwdWorks works = bwd_works(N, n_heads, a.Hkv, f);
  TP_RETURN_IF(ready());
  a.err = device_error_word();
  a.QKV = QKV;
  a.lse = const_cast<float*>(lse);
  a.O = const_cast<uint16_t*>(O);
  a.dO = dO;
  a.Dvec = Dvec;
  a.dQKV = dQKV;
  a.dqkv_f16 = dqkv_f16;
  a.wide = (reinterpret_cast<uintptr_t>(dQKV) & 31u) == 0;
  a.C = f.C;
  a.nch = f.nch;
  a.nsb = f.nsb;
  a.nfar = static_cast<int>(works.far);
  a.far = reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + span_bytes(N, o.n_seq));
  CUtensorMap m_qkv, m_do;
  if (!make_map_3d_bf16(&m_qkv, QKV, sh.row_w, N, t, sh.row_w * 2, N * sh.row_w * 2, 64, 64) ||
      !make_map_3d_bf16(&m_do, dO, sh.dt, N, t, sh.dt * 2, N * sh.dt * 2, 64, 64))
    return TP_FAIL_DETAIL("cuTensorMapEncodeTiled failed for QKV or dO");
  static bool configured[64] = {};
  int dev = 0;
  TP_CUDA_CHECK(cudaGetDevice(&dev));
  if (dev < 0 || dev >= 64) return TP_ERR_CUDA;
  if (!configured[dev]) {
    TP_CUDA_CHECK(cudaFuncSetAttribute(window_dkv_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, DKV_SMEM));
    TP_CUDA_CHECK(cudaFuncSetAttribute(window_dq_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, DQ_SMEM));
    configured[dev] = true;
  }
  int* total = o.n_seq > 0 ? static_cast<int*>(ws) : nullptr;
  int2* span = o.n_seq > 0 ? reinterpret_cast<int2*>(static_cast<uint8_t*>(ws) + 256) : nullptr;
  TP_CUDA_CHECK(launch_pdl(window_prep_kernel, dim3(static_cast<unsigned>(works.kv)), dim3(PREP_THREADS), 0, s, a,
                           o.cu_seqlens, static_cast<int>(o.n_seq), total, span));
  count_launch();
  a.total = total;
  a.span = span;
  TP_CUDA_CHECK(launch_pdl(window_dq_kernel, dim3(static_cast<unsigned>(works.q)), dim3(DQ_THREADS), DQ_SMEM, s, m_qkv,
                           m_do, a));
  count_launch();
  TP_CUDA_CHECK(launch_pdl(window_dkv_kernel, dim3(static_cast<unsigned>(works.far + works.kv)), dim3(BWD_THREADS), DKV_SMEM,
                           s, m_qkv, m_do, a));
  count_launch();
  if (works.far > 0) {
    TP_CUDA_CHECK(launch_pdl(window_sink_kernel, dim3(static_cast<unsigned>(works.kv)), dim3(SINK_THREADS), 0, s, a));
    count_launch();
  }
  return TP_OK;
}

}  // namespace tp
