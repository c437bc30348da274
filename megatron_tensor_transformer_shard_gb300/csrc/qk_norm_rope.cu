// RMS norm of every query and key head and the rotary position embedding, in one pass over
// the QKV rows of the sharded attention block ([t][N][R], a shard's row [its query heads | its
// K heads | its V heads], 128 columns a head; "02 — Tensor Parallelism", "The attention
// pairing": heads are independent, so both act on a shard's own heads without communication).
//
// For a head's 128 values x at position p, with gamma the head norm's weight (one vector for
// all query heads, one for all key heads) and f_i the frequency of pair i < rot / 2:
//   r = (mean(x^2) + eps)^-1/2,   u = r gamma x,
//   y_a = u_a cos(p f_i) - u_b sin(p f_i),  y_b = u_a sin(p f_i) + u_b cos(p f_i),
// (a, b) = (i, i + rot / 2), or (2 i, 2 i + 1) interleaved; columns from rot on keep u.
// Backward, with g = R^T dy:  dgamma = sum g r x,  dx = r (g gamma - x r^2 mean(g gamma x)).
//
// What bounds it: HBM.  A row is read once and written once, so the instructions must stay
// under the ~23 cycles (90 issue slots) an SM has per 512 bytes of head traffic.  Sixteen lanes
// hold one head, 4 pairs each: a lane loads both halves of its pairs (two 8-byte pieces rot / 2
// columns apart, or one 16-byte piece interleaved), so the rotation needs no exchange between
// lanes and four angles a lane.  (With 8 consecutive columns a lane the partner half came by
// shuffles, with eight angles a lane and a selection between query and key factors per element:
// 1330 us for 32768 tokens, 64 / 8 heads, forward and backward, against 720; the copies through
// shared memory below bring that to 563.)  A token's sines and cosines are formed once and
// multiplied by gamma once for the query heads and once for the key heads.  Arithmetic is
// packed, two fp32 an instruction.
//
// Angles: p f_i is needed modulo a turn, and for p in the 10^5s an fp32 product would be off by
// 10^-2.  f_i / 2 pi is kept as a 64-bit fraction of a turn (rounded from fp64), so the
// integer product with p, modulo 2^64, is the phase with no error beyond |p| 2^-54 turns at any
// 32-bit position; its top 32 bits feed sincospif.  The fractions are formed once per CTA
// (fp64 is slow here) and kept in shared memory.
#include <cuda_runtime.h>

#include <cmath>

#include "attn_tiles.cuh"
#include "decode_plan.cuh"
#include "devmath.cuh"
#include "internal.h"
#include "ptx.cuh"

namespace tp {
namespace {

constexpr int LANES = 16;                  // lanes that hold one head
constexpr int THREADS = 256;
constexpr int GROUPS = THREADS / LANES;    // 16-lane groups of a CTA

struct QkArgs {
  const uint16_t* x;        // [t][N][R]
  int64_t x_shard, x_row;   // append: elements from a shard, a row of x to the next
  uint16_t* y;              // rows: [t][N][R]; append: Q [N][n_heads][128]
  int64_t rows, N, R;       // rows = t N
  int q_t, kv_t, nh;        // heads of a shard: query, KV; heads walked (with or without the V heads)
  int hpg, chunks;          // heads per group visit, visits per row
  const uint16_t *q_gamma, *k_gamma;
  float eps;
  const double* inv_freq;
  int rot;
  const int32_t* pos;
  // append
  uint16_t *Kc, *Vc;        // [t][kv_t][N][L_max][128]
  int64_t L_max, window, n_sink;
  int rolling, n_heads;
  int* err;
  uint64_t timeout_ns;
  // backward
  const uint16_t* dy;       // [t][N][R]
  float* part;              // [gridDim.x][2][128] sums for dq_gamma, dk_gamma
};

enum : int { ROT_NONE = 0, ROT_HALF = 1, ROT_INTER = 2 };

// 1 / 2 pi in the frequencies' turns; see the top.
__device__ __forceinline__ uint64_t turn_fraction(double f) {
  const double v = f * 0.15915494309189535;
  return __double2ull_rn((v - floor(v)) * 18446744073709551616.0);
}

// Frequencies of the rot / 2 pairs as turn fractions in shared memory, by every thread of the CTA.
template <int ROT>
__device__ __forceinline__ void load_fractions(const QkArgs& a, uint64_t* frac) {
  if (ROT == ROT_NONE) return;
  if (threadIdx.x < HD / 2 && static_cast<int>(threadIdx.x) < a.rot / 2)
    frac[threadIdx.x] = turn_fraction(a.inv_freq[threadIdx.x]);
  __syncthreads();
}

__device__ __forceinline__ void sincos_at(uint64_t frac, int32_t p, float& s, float& c) {
  const uint64_t phase = frac * static_cast<uint64_t>(static_cast<int64_t>(p));
  // top 32 bits, rounded, as a signed fraction of half a turn
  const int32_t top = static_cast<int32_t>(static_cast<uint32_t>((phase + 0x80000000ull) >> 32));
  sincospif(static_cast<float>(top) * 4.656612873077393e-10f, &s, &c);
}

// Eight values of a head as 4 pairs (a_k, b_k), two pairs a packed word.
struct Pairs {
  uint64_t a[2], b[2];
};

// Where a lane's values lie in a head's 128 columns: pieces of 4 columns at c0 and c1.  ROT_HALF:
// lanes below rot / 8 hold the pairs 4 l .. 4 l + 3 (columns 4 l and rot / 2 + 4 l), the others 8
// columns behind rot; else columns 8 l .. 8 l + 7, whose pairs are neighbours when interleaved.
template <int ROT>
struct LaneCols {
  int c0, c1;
  __device__ LaneCols(int lane, int rot) {
    c0 = 8 * lane;
    c1 = c0 + 4;
    if (ROT == ROT_HALF && 8 * lane < rot) {
      c0 = 4 * lane;
      c1 = rot / 2 + c0;
    }
  }
  __device__ uint4 load(const uint16_t* head) const {
    if (ROT != ROT_HALF) return *reinterpret_cast<const uint4*>(head + c0);
    const uint2 x = *reinterpret_cast<const uint2*>(head + c0), y = *reinterpret_cast<const uint2*>(head + c1);
    return make_uint4(x.x, x.y, y.x, y.y);
  }
  __device__ void store(uint16_t* head, const uint4& w) const {
    if (ROT != ROT_HALF) {
      *reinterpret_cast<uint4*>(head + c0) = w;
      return;
    }
    *reinterpret_cast<uint2*>(head + c0) = make_uint2(w.x, w.y);
    *reinterpret_cast<uint2*>(head + c1) = make_uint2(w.z, w.w);
  }
  // column of a_k (which = 0) or b_k (which = 1)
  __device__ int col(int k, int which) const {
    if (ROT == ROT_INTER) return c0 + 2 * k + which;
    return (which ? c1 : c0) + k;
  }
};

template <int ROT, bool BF16>
__device__ __forceinline__ Pairs to_pairs(const uint4& w) {
  float v[8];
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    if (BF16) unpack_bf16x2(u[k], v[2 * k], v[2 * k + 1]);
    else unpack_f16x2(u[k], v[2 * k], v[2 * k + 1]);
  }
  Pairs p;
  if (ROT == ROT_INTER) {
    p.a[0] = f2_pack(v[0], v[2]);
    p.a[1] = f2_pack(v[4], v[6]);
    p.b[0] = f2_pack(v[1], v[3]);
    p.b[1] = f2_pack(v[5], v[7]);
  } else {
    p.a[0] = f2_pack(v[0], v[1]);
    p.a[1] = f2_pack(v[2], v[3]);
    p.b[0] = f2_pack(v[4], v[5]);
    p.b[1] = f2_pack(v[6], v[7]);
  }
  return p;
}
template <int ROT, bool BF16>
__device__ __forceinline__ uint4 from_pairs(const Pairs& p) {
  float a[4], b[4];
  f2_unpack(p.a[0], a[0], a[1]);
  f2_unpack(p.a[1], a[2], a[3]);
  f2_unpack(p.b[0], b[0], b[1]);
  f2_unpack(p.b[1], b[2], b[3]);
  auto two = [](float x, float y) { return BF16 ? pack_bf16x2(x, y) : pack_f16x2(x, y); };
  if (ROT == ROT_INTER) return make_uint4(two(a[0], b[0]), two(a[1], b[1]), two(a[2], b[2]), two(a[3], b[3]));
  return make_uint4(two(a[0], a[1]), two(a[2], a[3]), two(b[0], b[1]), two(b[2], b[3]));
}

// cos and sin of a lane's four angles at position p (1, 0 where it holds no rotated pair).
template <int ROT>
__device__ __forceinline__ void lane_angles(const QkArgs& a, const uint64_t* frac, int lane, int32_t p, uint64_t (&c2)[2],
                                            uint64_t (&s2)[2]) {
  float c[4] = {1.f, 1.f, 1.f, 1.f}, s[4] = {0.f, 0.f, 0.f, 0.f};
  if (ROT != ROT_NONE && 8 * lane < a.rot) {
#pragma unroll
    for (int k = 0; k < 4; ++k) sincos_at(frac[4 * lane + k], p, s[k], c[k]);
  }
  c2[0] = f2_pack(c[0], c[1]);
  c2[1] = f2_pack(c[2], c[3]);
  s2[0] = f2_pack(s[0], s[1]);
  s2[1] = f2_pack(s[2], s[3]);
}

__device__ __forceinline__ uint64_t f2_neg(uint64_t x) { return x ^ 0x8000000080000000ull; }
__device__ __forceinline__ float f2_sum(uint64_t x) {
  float a, b;
  f2_unpack(x, a, b);
  return a + b;
}

// Sum over the 16 lanes of a group (every lane gets it, in the same order).  Both groups of a warp
// take part: with a mask of one group's lanes the compiler orders every shuffle by a warp barrier.
__device__ __forceinline__ float group_sum(float v) {
#pragma unroll
  for (int o = LANES / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// r = 1 / rms of a head.  A sum of squares that leaves fp32 at the top (|x| above 10^18), or one that
// loses bits at the bottom with an eps no larger (below 2^-100 together), is formed again from values
// scaled by 2^-64 or 2^64, and x is left scaled with r to match, so that every finite bf16 row gets its
// result (at the top eps is far below such a row's mean square); r_true is 1 / rms.  Zeros with eps = 0
// have r = 0: they stay zeros and get no gradient.
__device__ __forceinline__ float inv_rms(Pairs& x, float eps, float& r_true) {
  auto squares = [&]() {
    return f2_fma(x.a[0], x.a[0], f2_fma(x.a[1], x.a[1], f2_fma(x.b[0], x.b[0], f2_mul(x.b[1], x.b[1]))));
  };
  const float ss = group_sum(f2_sum(squares()));
  const float ms = fmaf(ss, 1.0f / HD, eps);
  float r = r_true = rsqrtf(ms);
  const bool over = ss > 3.0e38f, under = ms < 7.9e-31f;
  if (__any_sync(0xffffffffu, over || under)) {
    const float d = over ? 5.42101086e-20f : under ? 18446744073709551616.0f : 1.0f;  // 2^-64, 2^64
    const uint64_t scaled = f2_pack(d, d);
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      x.a[k] = f2_mul(x.a[k], scaled);
      x.b[k] = f2_mul(x.b[k], scaled);
    }
    const float s2 = group_sum(f2_sum(squares()));
    if (over || under) {
      const float m2 = over ? s2 * (1.0f / HD) : fmaf(s2, 1.0f / HD, eps * d * d);
      r = m2 > 0.0f ? rsqrtf(m2) : 0.0f;
      r_true = fminf(r * d, 3.4e38f);  // finite, as it may meet a 0
    }
  }
  return r;
}

// The work of a 16-lane group's visit: row (shard, token n), heads [h0, h1).
struct Visit {
  int64_t row, shard, n;
  int h0, h1;
  int32_t p;
  __device__ Visit(const QkArgs& a, int64_t u) {
    row = u / a.chunks;
    h0 = static_cast<int>(u - row * a.chunks) * a.hpg;
    h1 = min(h0 + a.hpg, a.nh);
    shard = row / a.N;
    n = row - shard * a.N;
    p = a.pos ? a.pos[n] : static_cast<int32_t>(n);
  }
};

// The decode form: few rows, whose results go to other places.  A 16-lane group per (row, run of heads).
template <bool BF16, int ROT, bool NORM>
__global__ void __launch_bounds__(THREADS, 2) qk_norm_rope_append_kernel(const QkArgs a) {
  __shared__ uint64_t frac[HD / 2];
  ptx::griddep_wait();  // the rows, positions and parameters may come from the previous kernel
  ptx::griddep_launch_dependents();
  const int lane = threadIdx.x & 15;
  const LaneCols<ROT> cols(lane, a.rot);
  const int64_t units = a.rows * a.chunks;
  const int64_t stride = static_cast<int64_t>(gridDim.x) * GROUPS;
  const int64_t first = static_cast<int64_t>(blockIdx.x) * GROUPS + threadIdx.x / LANES;
  // A head is loaded while the one before is worked on, and a visit's first beside its position; the first of
  // all beside the frequencies (256 tokens, 64 / 8 heads, cold L2: 17.5 -> 15.5 us with the launch).
  auto head = [&](const Visit& v, int h) {
    const bool here = h < v.h1;
    return here ? cols.load(a.x + v.shard * a.x_shard + v.n * a.x_row + static_cast<int64_t>(h) * HD)
                : make_uint4(0u, 0u, 0u, 0u);
  };
  int64_t u0 = first & ~static_cast<int64_t>(1);
  Visit v(a, min(u0 + (first & 1), units - 1));
  uint4 next = head(v, v.h0);
  const Pairs qg = NORM ? to_pairs<ROT, true>(cols.load(a.q_gamma)) : Pairs{};
  const Pairs kg = NORM ? to_pairs<ROT, true>(cols.load(a.k_gamma)) : Pairs{};
  load_fractions<ROT>(a, frac);
  // both groups of a warp stay in every loop together (the reductions shuffle warp-wide)
  for (; u0 < units; u0 += stride) {
    const int64_t u = u0 + (first & 1);
    if (u0 != (first & ~static_cast<int64_t>(1))) {
      v = Visit(a, min(u, units - 1));
      next = head(v, v.h0);
    }
    const bool on = u < units && v.p >= 0;
    int64_t slot = -1;  // of the caches, -1 for none
    // a negative position other than -1, or one past the cache, is an argument error
    if (v.p >= 0) {
      slot = v.p;
      if (a.rolling && v.p >= a.n_sink + a.window) slot = a.n_sink + (v.p - a.n_sink) % a.window;
      if (slot >= a.L_max) slot = -1;
    }
    if (lane == 0 && (v.p < -1 || (v.p >= 0 && slot < 0))) atomicCAS(a.err, 0, kDecodeErrPos);
    uint64_t c2[2], s2[2];
    lane_angles<ROT>(a, frac, lane, v.p, c2, s2);
    const int64_t kv_stride = a.N * a.L_max * HD;
    const int64_t kv0 = ((v.shard * a.kv_t * a.N + v.n) * a.L_max + slot) * HD;  // the slot in the shard's first KV head
    for (int i = 0; i < a.hpg; ++i) {
      const int h = v.h0 + i;
      const bool here = on && h < v.h1;
      const uint4 w = next;
      if (i + 1 < a.hpg) next = head(v, h + 1);
      const bool is_q = h < a.q_t, is_v = h >= a.q_t + a.kv_t;
      Pairs x = to_pairs<ROT, BF16>(w), y;
      const Pairs raw = x;
      float r = 1.0f, r_true;
      if (NORM) r = inv_rms(x, a.eps, r_true);
      const uint64_t r2 = f2_pack(r, r);
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        // the order of roundings is that of the rows' kernel: the same bits
        const uint64_t ga = is_q ? qg.a[k] : kg.a[k], gb = is_q ? qg.b[k] : kg.b[k];
        const uint64_t faa = NORM ? f2_mul(c2[k], ga) : c2[k], fba = NORM ? f2_mul(s2[k], ga) : s2[k];
        const uint64_t fab = NORM ? f2_mul(f2_neg(s2[k]), gb) : f2_neg(s2[k]), fbb = NORM ? f2_mul(c2[k], gb) : c2[k];
        y.a[k] = ROT == ROT_NONE ? f2_mul(x.a[k], faa) : f2_fma(x.b[k], fab, f2_mul(x.a[k], faa));
        y.b[k] = ROT == ROT_NONE ? f2_mul(x.b[k], fbb) : f2_fma(x.b[k], fbb, f2_mul(x.a[k], fba));
        if (NORM) {
          y.a[k] = f2_mul(y.a[k], r2);
          y.b[k] = f2_mul(y.b[k], r2);
        }
      }
      const uint4 o = is_v ? (BF16 ? from_pairs<ROT, false>(raw) : w) : from_pairs<ROT, false>(y);
      if (here && is_q) {
        cols.store(a.y + (v.n * a.n_heads + v.shard * a.q_t + h) * HD, o);
      } else if (here && slot >= 0) {
        uint16_t* cache = is_v ? a.Vc : a.Kc;
        cols.store(cache + kv0 + (h - a.q_t - (is_v ? a.kv_t : 0)) * kv_stride, o);
      }
    }
  }
}

// ------------------------------------------------------------ rows through shared memory
//
// Forward and backward over many rows.  With loads into registers the kernels had 32 KB of reads
// in flight an SM, less than HBM latency times an SM's share of the bandwidth, and the registers
// for more cost the occupancy that hid the arithmetic.  So each warp streams its own units (a
// run of heads of one token's row, contiguous in memory) through a private ring of STREAM_RING
// slots: bulk copies in, the arithmetic in place in shared memory, bulk copies out of the same
// slot, one load ahead.  No barrier between warps.  Units run token-major (token, shard, run of
// heads), each warp over a contiguous range of them, so the sines and cosines of a token are
// formed once for all its shards' heads, by all 32 lanes, and wait in shared memory.
// Measured (N 32768, 64 / 8 heads, t 8, norm + rotation): forward 238 us = 5.6 TB/s, 85 % of the
// copy rate; backward 335 us = 5.8 TB/s of dY, X, dX, 87 % (55 % of the issue slots taken); both, one
// after the other, 563 us; the register version 720.  96 heads x 2048: both 121 us (87 % of the copy rate).
constexpr int STREAM_WARPS = 12, STREAM_THREADS = STREAM_WARPS * 32, STREAM_RING = 3;
constexpr int WARP_EXTRA = 2 * (HD / 2) * 4 + 64;  // cosines, sines, ring barriers
constexpr size_t SUMS_BYTES = 2 * STREAM_WARPS * 2 * HD * sizeof(float);  // dgamma of two groups a warp
enum : int { ERR_QKNR_STREAM = 0x161 };

// Position in the unit order of one warp.
struct UnitCursor {
  int n, shard, chunk;
  __device__ UnitCursor(const QkArgs& a, int64_t u) {
    chunk = static_cast<int>(u % a.chunks);
    u /= a.chunks;
    const int t = static_cast<int>(a.rows / a.N);
    shard = static_cast<int>(u % t);
    n = static_cast<int>(u / t);
  }
  __device__ void next(const QkArgs& a, int t) {
    if (++chunk < a.chunks) return;
    chunk = 0;
    if (++shard < t) return;
    shard = 0;
    ++n;
  }
  __device__ int h0(const QkArgs& a) const { return chunk * a.hpg; }
  __device__ int h1(const QkArgs& a) const { return min(chunk * a.hpg + a.hpg, a.nh); }
  __device__ int64_t offset(const QkArgs& a) const {  // of the unit's first value in [t][N][R]
    return (static_cast<int64_t>(shard) * a.N + n) * a.R + static_cast<int64_t>(h0(a)) * HD;
  }
};

// The 64 cosines and sines of position p into the warp's table (1, 0 behind the rotated pairs).
template <int ROT>
__device__ __forceinline__ void fill_table(const QkArgs& a, const uint64_t* frac, float* cs, int32_t p) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const int i = lane + 32 * k;
    float s = 0.0f, c = 1.0f;
    if (i < a.rot / 2) sincos_at(frac[i], p, s, c);
    cs[i] = c;
    cs[HD / 2 + i] = s;
  }
  __syncwarp();
}
__device__ __forceinline__ void read_table(const float* cs, int lane, uint64_t (&c2)[2], uint64_t (&s2)[2]) {
  const float4 c = *reinterpret_cast<const float4*>(cs + 4 * lane), s = *reinterpret_cast<const float4*>(cs + HD / 2 + 4 * lane);
  c2[0] = f2_pack(c.x, c.y);
  c2[1] = f2_pack(c.z, c.w);
  s2[0] = f2_pack(s.x, s.y);
  s2[1] = f2_pack(s.z, s.w);
}

// BWD: a slot holds the unit's dY, then its X (query and key heads); dX replaces dY.
template <bool BWD, bool BF16, bool GBF16, int ROT, bool NORM>
__global__ void __launch_bounds__(STREAM_THREADS, 1) qk_norm_rope_stream_kernel(const QkArgs a, int slot_bytes) {
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ uint64_t frac[HD / 2];
  __shared__ int abort_flag;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  uint8_t* mine = smem + warp * (STREAM_RING * slot_bytes + WARP_EXTRA);
  float* cs = reinterpret_cast<float*>(mine + STREAM_RING * slot_bytes);
  uint64_t* full = reinterpret_cast<uint64_t*>(cs + HD);
  if (lane == 0) {
    for (int s = 0; s < STREAM_RING; ++s) ptx::mbar_init(&full[s], 1);
    ptx::fence_mbar_init();
  }
  if (threadIdx.x == 0) abort_flag = 0;
  ptx::griddep_wait();  // the rows, positions and parameters may come from the previous kernel
  ptx::griddep_launch_dependents();
  load_fractions<ROT>(a, frac);
  __syncthreads();
  const int t = static_cast<int>(a.rows / a.N);
  const int64_t units = a.rows * a.chunks;
  // warps of all CTAs, CTA by CTA within a rank: few units go to different SMs
  const int64_t w = static_cast<int64_t>(warp) * gridDim.x + blockIdx.x, W = static_cast<int64_t>(gridDim.x) * STREAM_WARPS;
  const int64_t u0 = w * units / W;
  const int count = static_cast<int>((w + 1) * units / W - u0);
  const int nqk = a.q_t + a.kv_t;

  UnitCursor ahead(a, u0), cur = ahead;
  auto load = [&](int i) {  // lane 0: unit i's bytes into its slot
    const int h0 = ahead.h0(a), h1 = ahead.h1(a), x1 = min(h1, nqk);
    const int64_t at = ahead.offset(a);
    uint8_t* dst = mine + (i % STREAM_RING) * slot_bytes;
    uint64_t* bar = &full[i % STREAM_RING];
    const uint32_t bytes = (h1 - h0) * HD * 2, xbytes = BWD && NORM && x1 > h0 ? (x1 - h0) * HD * 2 : 0;
    ptx::mbar_arrive_expect_tx(bar, bytes + xbytes);
    ptx::bulk_load(dst, (BWD ? a.dy : a.x) + at, bytes, bar);
    if (xbytes) ptx::bulk_load(dst + slot_bytes / 2, a.x + at, xbytes, bar);
  };
  if (lane == 0) {
    for (int i = 0; i < STREAM_RING - 2 && i < count; ++i) {
      load(i);
      ahead.next(a, t);
    }
  }

  const int gl = lane & 15, grp = lane >> 4;
  const LaneCols<ROT> cols(gl, a.rot);
  Pairs qg{}, kg{}, dq{}, dk{};
  if (NORM) {
    qg = to_pairs<ROT, true>(cols.load(a.q_gamma));
    kg = to_pairs<ROT, true>(cols.load(a.k_gamma));
  }
  int n_table = -1;
  int32_t p_next = count > 0 && a.pos ? a.pos[cur.n] : 0;
  for (int i = 0; i < count; ++i) {
    if (lane == 0 && i + STREAM_RING - 2 < count) {
      ptx::bulk_wait_group_read<1>();  // unit i - 2 has left the slot
      load(i + STREAM_RING - 2);
      ahead.next(a, t);
    }
    if (ROT != ROT_NONE && cur.n != n_table) {
      n_table = cur.n;
      __syncwarp();  // every lane is done with the old table
      fill_table<ROT>(a, frac, cs, a.pos ? p_next : n_table);
      if (a.pos && n_table + 1 < a.N) p_next = a.pos[n_table + 1];
    }
    uint64_t c2[2], s2[2];
    if (ROT == ROT_NONE) {
      c2[0] = c2[1] = f2_pack(1.0f, 1.0f);
      s2[0] = s2[1] = 0;
    } else {
      read_table(cs, gl, c2, s2);
    }
    uint16_t* slot = reinterpret_cast<uint16_t*>(mine + (i % STREAM_RING) * slot_bytes);
    uint16_t* xslot = slot + slot_bytes / 4;
    const bool here = ptx::mbar_wait(&full[i % STREAM_RING], (i / STREAM_RING) & 1, &abort_flag, a.err, ERR_QKNR_STREAM,
                                     a.timeout_ns);
    if (!__all_sync(0xffffffffu, here)) {
      volatile int never = 0;  // the copies in flight land before the CTA exits
      for (int k = i; lane == 0 && k < min(i + STREAM_RING - 1, count); ++k)
        ptx::mbar_wait(&full[k % STREAM_RING], (k / STREAM_RING) & 1, &never, a.err, ERR_QKNR_STREAM, a.timeout_ns);
      break;
    }
    const int h0 = cur.h0(a), h1 = cur.h1(a);

    // Heads [ha, hb) of one kind, two at a time: the lower 16 lanes one, the upper the next (zeros, and
    // nothing stored, behind the last).
    auto heads = [&](int ha, int hb, const Pairs& gam, Pairs& dg) {
      if (ha >= hb) return;
      uint64_t faa[2], fab[2], fba[2], fbb[2];  // y_a = a faa + b fab, y_b = a fba + b fbb, gamma folded in
      if (!BWD) {
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          faa[k] = NORM ? f2_mul(c2[k], gam.a[k]) : c2[k];
          fba[k] = NORM ? f2_mul(s2[k], gam.a[k]) : s2[k];
          fab[k] = NORM ? f2_mul(f2_neg(s2[k]), gam.b[k]) : f2_neg(s2[k]);
          fbb[k] = NORM ? f2_mul(c2[k], gam.b[k]) : c2[k];
        }
      }
#pragma unroll 2
      for (int h = ha; h < hb; h += 2) {
        const bool on = h + grp < hb;
        uint16_t* head = slot + (h + grp - h0) * HD;
        const uint4 w = on ? cols.load(head) : make_uint4(0u, 0u, 0u, 0u);
        if (!BWD) {
          Pairs x = to_pairs<ROT, BF16>(w), y;
          float r = 1.0f, r_true;
          if (NORM) r = inv_rms(x, a.eps, r_true);
          const uint64_t r2 = f2_pack(r, r);
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            if (ROT == ROT_NONE) {
              y.a[k] = f2_mul(x.a[k], faa[k]);
              y.b[k] = f2_mul(x.b[k], fbb[k]);
            } else {
              y.a[k] = f2_fma(x.b[k], fab[k], f2_mul(x.a[k], faa[k]));
              y.b[k] = f2_fma(x.b[k], fbb[k], f2_mul(x.a[k], fba[k]));
            }
            if (NORM) {
              y.a[k] = f2_mul(y.a[k], r2);
              y.b[k] = f2_mul(y.b[k], r2);
            }
          }
          const uint4 o = from_pairs<ROT, false>(y);
          if (on) cols.store(head, o);
        } else {
          const Pairs d = to_pairs<ROT, GBF16>(w);
          Pairs g = d;
          if (ROT != ROT_NONE) {  // the transposed rotation
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              g.a[k] = f2_fma(d.b[k], s2[k], f2_mul(d.a[k], c2[k]));
              g.b[k] = f2_fma(d.a[k], f2_neg(s2[k]), f2_mul(d.b[k], c2[k]));
            }
          }
          if (NORM) {
            Pairs x = to_pairs<ROT, BF16>(on ? cols.load(xslot + (h + grp - h0) * HD) : make_uint4(0u, 0u, 0u, 0u));
            float r_true;
            const float r = inv_rms(x, a.eps, r_true);
            const uint64_t r2 = f2_pack(r, r), out2 = f2_pack(r_true, r_true);
            uint64_t dot2 = 0;
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              x.a[k] = f2_mul(x.a[k], r2);  // the normalised input
              x.b[k] = f2_mul(x.b[k], r2);
              dg.a[k] = f2_fma(g.a[k], x.a[k], dg.a[k]);
              dg.b[k] = f2_fma(g.b[k], x.b[k], dg.b[k]);
              g.a[k] = f2_mul(g.a[k], gam.a[k]);
              g.b[k] = f2_mul(g.b[k], gam.b[k]);
              dot2 = f2_fma(g.a[k], x.a[k], dot2);
              dot2 = f2_fma(g.b[k], x.b[k], dot2);
            }
            const float dot = group_sum(f2_sum(dot2)) * (-1.0f / HD);
            const uint64_t nd = f2_pack(dot, dot);
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              g.a[k] = f2_mul(out2, f2_fma(x.a[k], nd, g.a[k]));
              g.b[k] = f2_mul(out2, f2_fma(x.b[k], nd, g.b[k]));
            }
          }
          const uint4 o = from_pairs<ROT, GBF16>(g);
          if (on) cols.store(head, o);
        }
      }
    };
    const int q1 = min(h1, a.q_t), k0 = max(h0, a.q_t), k1 = min(h1, nqk);
    heads(h0, q1, qg, dq);
    heads(k0, k1, kg, dk);
    if (!BWD && BF16) {  // the values are carried over
      for (int e = max(h0, nqk) * 16 + lane; e < h1 * 16; e += 32) {
        uint4* v = reinterpret_cast<uint4*>(slot) + (e - h0 * 16);
        *v = from_pairs<ROT_NONE, false>(to_pairs<ROT_NONE, true>(*v));
      }
    }
    ptx::fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) {
      ptx::bulk_store(a.y + cur.offset(a), slot, (h1 - h0) * HD * 2);
      ptx::bulk_commit_group();
    }
    cur.next(a, t);
  }
  if (lane == 0) ptx::bulk_wait_group<0>();

  if (BWD && NORM) {
    // dgamma: a lane has added its 8 columns over the heads it visited (fp32 registers); the CTA's
    // groups are added in order, the CTAs' sums in CTA order by the next kernel, so the result does
    // not depend on timing.
    __syncthreads();  // the rings are done with
    float* sums = reinterpret_cast<float*>(smem);  // SUMS_BYTES: [24 groups][2][128]
    const int group = warp * 2 + grp;
#pragma unroll
    for (int kind = 0; kind < 2; ++kind) {
      const Pairs& d = kind ? dk : dq;
      float* row = sums + (group * 2 + kind) * HD;
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        float v0, v1;
        f2_unpack(d.a[k], v0, v1);
        row[cols.col(2 * k, 0)] = v0;
        row[cols.col(2 * k + 1, 0)] = v1;
        f2_unpack(d.b[k], v0, v1);
        row[cols.col(2 * k, 1)] = v0;
        row[cols.col(2 * k + 1, 1)] = v1;
      }
    }
    __syncthreads();
    if (threadIdx.x < 2 * HD) {
      float v = 0.0f;
#pragma unroll 8
      for (int k = 0; k < 2 * STREAM_WARPS; ++k) v += sums[k * 2 * HD + threadIdx.x];
      a.part[static_cast<int64_t>(blockIdx.x) * 2 * HD + threadIdx.x] = v;
    }
  }
}

// dgamma = the CTAs' sums in CTA order: 16 columns a CTA, 64 threads a column, each over every 64th sum.
constexpr int FIN_COLS = 16, FIN_ROWS = 64;
__global__ void __launch_bounds__(FIN_COLS * FIN_ROWS)
    dgamma_final_kernel(const float* part, int G, float* dq_gamma, float* dk_gamma, int accumulate) {
  __shared__ float s[FIN_ROWS][FIN_COLS + 1];
  ptx::griddep_wait();
  ptx::griddep_launch_dependents();
  const int c = threadIdx.x % FIN_COLS, r = threadIdx.x / FIN_COLS;
  const int col = blockIdx.x * FIN_COLS + c;
  float v = 0.0f;
  for (int k = r; k < G; k += FIN_ROWS) v += part[static_cast<int64_t>(k) * 2 * HD + col];
  s[r][c] = v;
  __syncthreads();
  for (int o = FIN_ROWS / 2; o > 0; o >>= 1) {
    if (r < o) s[r][c] += s[r + o][c];
    __syncthreads();
  }
  if (r == 0) {
    float* out = col < HD ? dq_gamma : dk_gamma;
    if (out) {
      out += col & (HD - 1);
      *out = accumulate ? *out + s[0][c] : s[0][c];
    }
  }
}

// CTAs for `units` group visits, at most `per_sm` for each multiprocessor.
unsigned grid_for(int64_t units, int per_sm) {
  const int64_t want = (units + GROUPS - 1) / GROUPS;
  const int64_t most = static_cast<int64_t>(device_sm_count()) * per_sm;
  return static_cast<unsigned>(want < most ? (want > 0 ? want : 1) : most);
}

// Heads per group visit: all of a row's share the token's sines and cosines; few rows are cut finer, into
// at least 4 CTAs of 16 groups for each SM (two fit at a time).
void set_chunks(QkArgs& a) {
  const int64_t fill = static_cast<int64_t>(device_sm_count()) * 4 * GROUPS;
  int64_t chunks = (fill + a.rows - 1) / a.rows;
  if (chunks > a.nh) chunks = a.nh;
  a.hpg = static_cast<int>((a.nh + chunks - 1) / chunks);
  a.chunks = (a.nh + a.hpg - 1) / a.hpg;
}

template <bool BF16>
tp_status launch_append(const QkArgs& a, int rot, bool norm, unsigned grid, cudaStream_t s) {
  auto go = [&](auto kernel) -> tp_status {
    TP_CUDA_CHECK(launch_pdl(kernel, dim3(grid), dim3(THREADS), 0, s, a));
    count_launch();
    return TP_OK;
  };
  if (norm) {
    if (rot == ROT_NONE) return go(qk_norm_rope_append_kernel<BF16, ROT_NONE, true>);
    if (rot == ROT_HALF) return go(qk_norm_rope_append_kernel<BF16, ROT_HALF, true>);
    return go(qk_norm_rope_append_kernel<BF16, ROT_INTER, true>);
  }
  if (rot == ROT_NONE) return go(qk_norm_rope_append_kernel<BF16, ROT_NONE, false>);
  if (rot == ROT_HALF) return go(qk_norm_rope_append_kernel<BF16, ROT_HALF, false>);
  return go(qk_norm_rope_append_kernel<BF16, ROT_INTER, false>);
}

// Units of at most `most` heads; few rows are cut finer, so that every warp of the GPU gets some.
void set_units(QkArgs& a, int most) {
  int64_t chunks = (a.nh + most - 1) / most;
  const int64_t warps = static_cast<int64_t>(device_sm_count()) * STREAM_WARPS;
  if (a.rows * chunks < warps) chunks = (warps + a.rows - 1) / a.rows;
  if (chunks > a.nh) chunks = a.nh;
  a.hpg = static_cast<int>((a.nh + chunks - 1) / chunks);
  a.chunks = (a.nh + a.hpg - 1) / a.hpg;
}

// Heads of a unit at most (rings of up to 184 KB).  A unit costs about as many instructions around its
// heads (copies, cursors, waits) as two pairs of heads do, so whole rows beat more warps: backward units
// of 5 heads in 16 warps 625 us, of 10 in 12 warps 574 us (32768 tokens, 64 / 8 heads, both directions).
constexpr int FWD_HEADS = 12, BWD_HEADS = 10;
constexpr int BWD_MAX_GRID = 1024;            // the workspace has a sum for every CTA that any device may run

template <bool BWD, bool BF16, bool GBF16, int ROT, bool NORM>
tp_status launch_stream(const QkArgs& a, unsigned grid, cudaStream_t s) {
  auto kernel = qk_norm_rope_stream_kernel<BWD, BF16, GBF16, ROT, NORM>;
  const int slot = a.hpg * HD * 2 * (BWD && NORM ? 2 : 1);
  // the backward's last sums take the rings' room
  const size_t rings = static_cast<size_t>(STREAM_WARPS) * (STREAM_RING * slot + WARP_EXTRA);
  const size_t smem = BWD && NORM && rings < SUMS_BYTES ? SUMS_BYTES : rings;
  static bool configured[64] = {};
  int dev = 0;
  TP_CUDA_CHECK(cudaGetDevice(&dev));
  if (dev < 0 || dev >= 64) return TP_ERR_CUDA;
  if (!configured[dev]) {
    TP_CUDA_CHECK(cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 225 * 1024));
    configured[dev] = true;
  }
  TP_CUDA_CHECK(launch_pdl(kernel, dim3(grid), dim3(STREAM_THREADS), smem, s, a, slot));
  count_launch();
  return TP_OK;
}

template <bool BWD, bool BF16, bool GBF16>
tp_status launch_rows(QkArgs& a, int rot, bool norm, unsigned* grid_out, cudaStream_t s) {
  set_units(a, BWD && norm ? BWD_HEADS : FWD_HEADS);
  int64_t grid = device_sm_count();
  if (grid > a.rows * a.chunks) grid = a.rows * a.chunks;
  if (grid > BWD_MAX_GRID) grid = BWD_MAX_GRID;
  const unsigned g = static_cast<unsigned>(grid);
  if (grid_out) *grid_out = g;
  if (norm) {
    if (rot == ROT_NONE) return launch_stream<BWD, BF16, GBF16, ROT_NONE, true>(a, g, s);
    if (rot == ROT_HALF) return launch_stream<BWD, BF16, GBF16, ROT_HALF, true>(a, g, s);
    return launch_stream<BWD, BF16, GBF16, ROT_INTER, true>(a, g, s);
  }
  // without a norm there is a rotation, and the backward does not read the input
  if (rot == ROT_HALF) return launch_stream<BWD, BF16 && !BWD, GBF16, ROT_HALF, false>(a, g, s);
  return launch_stream<BWD, BF16 && !BWD, GBF16, ROT_INTER, false>(a, g, s);
}

// Checks shared by the three calls; fills the shape fields of `a`.
tp_status check_common(const QkNormRope& o, int64_t N, int n_heads, int n_kv, int head_dim, int t, QkArgs& a, int& rot,
                       bool& norm, bool copy_ok = false) {
  if (N < 0 || n_heads < 1 || n_kv < 1 || t < 1 || head_dim < 1) return TP_ERR_INVALID_ARG;
  if ((o.q_gamma == nullptr) != (o.k_gamma == nullptr)) return TP_ERR_INVALID_ARG;
  norm = o.q_gamma != nullptr;
  if (!norm && !o.inv_freq && !copy_ok) return TP_ERR_INVALID_ARG;
  if (norm && !(o.eps >= 0.0f && o.eps < INFINITY)) return TP_ERR_INVALID_ARG;
  if ((o.flags & ~(TP_QKNR_BF16_INPUT | TP_QKNR_F16_GRAD | TP_ROPE_INTERLEAVED)) != 0) return TP_ERR_UNSUPPORTED;
  if (head_dim != HD || n_heads % t != 0 || n_heads % n_kv != 0) return TP_ERR_SHAPE;
  if (n_kv >= t ? n_kv % t != 0 : t % n_kv != 0) return TP_ERR_SHAPE;
  rot = ROT_NONE;
  if (o.inv_freq) {
    if (o.rot_dim < 16 || o.rot_dim > HD || o.rot_dim % 16 != 0) return TP_ERR_SHAPE;
    rot = (o.flags & TP_ROPE_INTERLEAVED) ? ROT_INTER : ROT_HALF;
  }
  if (N > (1LL << 30)) return TP_ERR_SHAPE;
  if (!aligned16(o.q_gamma) || !aligned16(o.k_gamma) || (reinterpret_cast<uintptr_t>(o.inv_freq) & 7u) != 0 ||
      !aligned4(o.pos))
    return TP_ERR_ALIGN;
  a.N = N;
  a.rows = N * t;
  a.q_t = n_heads / t;
  a.kv_t = n_kv >= t ? n_kv / t : 1;
  a.nh = a.q_t + 2 * a.kv_t;
  a.R = static_cast<int64_t>(a.nh) * HD;
  a.n_heads = n_heads;
  a.q_gamma = o.q_gamma;
  a.k_gamma = o.k_gamma;
  a.eps = o.eps;
  a.inv_freq = o.inv_freq;
  a.rot = o.inv_freq ? o.rot_dim : 0;
  a.pos = o.pos;
  a.err = nullptr;
  return TP_OK;
}

// Ranges that share bytes without being the same range (in place is fine, partly over is not).
bool partly_over(const void* p, const void* q, size_t bytes) { return p != q && overlap(p, bytes, q, bytes); }

// All that a call can be refused for, before anything is launched; fills the shape fields of `a`.
tp_status check_fwd(const uint16_t* QKV, int64_t N, int n_heads, int n_kv, int head_dim, int t, const QkNormRope& o,
                    const uint16_t* out, QkArgs& a, int& rot, bool& norm) {
  TP_RETURN_IF(check_common(o, N, n_heads, n_kv, head_dim, t, a, rot, norm));
  if (o.flags & TP_QKNR_F16_GRAD) return TP_ERR_UNSUPPORTED;
  if (N == 0) return TP_OK;
  if (!QKV || !out) return TP_ERR_INVALID_ARG;
  if (!aligned16(QKV) || !aligned16(out)) return TP_ERR_ALIGN;
  if (partly_over(QKV, out, static_cast<size_t>(a.rows) * a.R * 2)) return TP_ERR_INVALID_ARG;
  return TP_OK;
}

tp_status check_append(const uint16_t* QKV, int64_t B, int n_heads, int n_kv, int head_dim, int t, const QkNormRope& o,
                       const uint16_t* Q, const uint16_t* Kc, const uint16_t* Vc, int64_t L_max, int64_t window,
                       int64_t n_sink, int rolling, int token_major, QkArgs& a, int& rot, bool& norm) {
  TP_RETURN_IF(check_common(o, B, n_heads, n_kv, head_dim, t, a, rot, norm, token_major != 0));
  if (o.flags & TP_QKNR_F16_GRAD) return TP_ERR_UNSUPPORTED;
  if (L_max < 1 || (rolling && (window < 1 || n_sink < 0))) return TP_ERR_INVALID_ARG;
  if (L_max > (1LL << 30)) return TP_ERR_SHAPE;
  if (rolling && (window > L_max || n_sink > L_max || n_sink + window > L_max)) return TP_ERR_SHAPE;
  if (B == 0) return TP_OK;
  if (!QKV || !Q || !Kc || !Vc || !o.pos) return TP_ERR_INVALID_ARG;
  if (!aligned16(QKV) || !aligned16(Q) || !aligned16(Kc) || !aligned16(Vc)) return TP_ERR_ALIGN;
  const size_t cache = static_cast<size_t>(t) * a.kv_t * B * L_max * HD * 2;
  const size_t qb = static_cast<size_t>(B) * n_heads * HD * 2;
  const size_t xb = static_cast<size_t>(a.rows) * a.R * 2;
  if (overlap(Kc, cache, Vc, cache) || overlap(Q, qb, Kc, cache) || overlap(Q, qb, Vc, cache) ||
      overlap(QKV, xb, Q, qb) || overlap(QKV, xb, Kc, cache) || overlap(QKV, xb, Vc, cache))
    return TP_ERR_INVALID_ARG;
  return TP_OK;
}

tp_status check_bwd(const uint16_t* dQKV, const uint16_t* QKV, int64_t N, int n_heads, int n_kv, int head_dim, int t,
                    const QkNormRope& o, const uint16_t* out, const float* dq_gamma, const float* dk_gamma, const void* ws,
                    size_t ws_bytes, QkArgs& a, int& rot, bool& norm) {
  TP_RETURN_IF(check_common(o, N, n_heads, n_kv, head_dim, t, a, rot, norm));
  if (!norm && (dq_gamma || dk_gamma)) return TP_ERR_INVALID_ARG;
  if (!aligned4(dq_gamma) || !aligned4(dk_gamma)) return TP_ERR_ALIGN;
  if (N == 0) return TP_OK;
  if (!dQKV || !out || (norm && !QKV)) return TP_ERR_INVALID_ARG;
  if (!aligned16(dQKV) || !aligned16(QKV) || !aligned16(out)) return TP_ERR_ALIGN;
  const size_t bytes = static_cast<size_t>(a.rows) * a.R * 2;
  if (partly_over(dQKV, out, bytes) || (norm && (QKV == out || partly_over(QKV, out, bytes)))) return TP_ERR_INVALID_ARG;
  if (norm && (!ws || ws_bytes < qk_norm_rope_bwd_ws_bytes())) return TP_ERR_WORKSPACE;
  if (norm && !aligned16(ws)) return TP_ERR_ALIGN;
  return TP_OK;
}

}  // namespace

size_t qk_norm_rope_bwd_ws_bytes() { return static_cast<size_t>(BWD_MAX_GRID) * 2 * HD * sizeof(float); }

tp_status qk_norm_rope_fwd_ok(const uint16_t* QKV, int64_t N, int n_heads, int n_kv, int head_dim, int t,
                              const QkNormRope& o, const uint16_t* out) {
  QkArgs a{};
  int rot;
  bool norm;
  return check_fwd(QKV, N, n_heads, n_kv, head_dim, t, o, out, a, rot, norm);
}

tp_status qk_norm_rope_append_ok(const uint16_t* QKV, int64_t B, int n_heads, int n_kv, int head_dim, int t,
                                 const QkNormRope& o, const uint16_t* Q, const uint16_t* Kc, const uint16_t* Vc,
                                 int64_t L_max, int64_t window, int64_t n_sink, int rolling, int token_major) {
  QkArgs a{};
  int rot;
  bool norm;
  return check_append(QKV, B, n_heads, n_kv, head_dim, t, o, Q, Kc, Vc, L_max, window, n_sink, rolling, token_major, a,
                      rot, norm);
}

tp_status qk_norm_rope_bwd_ok(const uint16_t* dQKV, const uint16_t* QKV, int64_t N, int n_heads, int n_kv, int head_dim,
                              int t, const QkNormRope& o, const uint16_t* out, const float* dq_gamma,
                              const float* dk_gamma, const void* ws, size_t ws_bytes) {
  QkArgs a{};
  int rot;
  bool norm;
  return check_bwd(dQKV, QKV, N, n_heads, n_kv, head_dim, t, o, out, dq_gamma, dk_gamma, ws, ws_bytes, a, rot, norm);
}

tp_status run_qk_norm_rope_fwd(const uint16_t* QKV, int64_t N, int n_heads, int n_kv, int head_dim, int t,
                               const QkNormRope& o, uint16_t* out, cudaStream_t s) {
  QkArgs a{};
  int rot;
  bool norm;
  TP_RETURN_IF(check_fwd(QKV, N, n_heads, n_kv, head_dim, t, o, out, a, rot, norm));
  if (N == 0) return TP_OK;
  TP_RETURN_IF(ready());
  const bool bf16 = (o.flags & TP_QKNR_BF16_INPUT) != 0;
  if (QKV == out && !bf16) a.nh = a.q_t + a.kv_t;  // in place: V stays as it is
  a.x = QKV;
  a.y = out;
  a.err = device_error_word();
  a.timeout_ns = wait_timeout_ns();
  return bf16 ? launch_rows<false, true, false>(a, rot, norm, nullptr, s)
              : launch_rows<false, false, false>(a, rot, norm, nullptr, s);
}

tp_status run_qk_norm_rope_append(const uint16_t* QKV, int64_t B, int n_heads, int n_kv, int head_dim, int t,
                                  const QkNormRope& o, uint16_t* Q, uint16_t* Kc, uint16_t* Vc, int64_t L_max,
                                  int64_t window, int64_t n_sink, int rolling, cudaStream_t s, int token_major) {
  QkArgs a{};
  int rot;
  bool norm;
  TP_RETURN_IF(check_append(QKV, B, n_heads, n_kv, head_dim, t, o, Q, Kc, Vc, L_max, window, n_sink, rolling, token_major,
                            a, rot, norm));
  if (B == 0) return TP_OK;
  TP_RETURN_IF(ready());
  a.x = QKV;
  a.x_shard = token_major ? a.R : B * a.R;
  a.x_row = token_major ? t * a.R : a.R;
  a.y = Q;
  a.Kc = Kc;
  a.Vc = Vc;
  a.L_max = L_max;
  a.window = window;
  a.n_sink = n_sink;
  a.rolling = rolling;
  a.err = device_error_word();
  set_chunks(a);
  const unsigned grid = grid_for(a.rows * a.chunks, 8);
  return (o.flags & TP_QKNR_BF16_INPUT) ? launch_append<true>(a, rot, norm, grid, s)
                                        : launch_append<false>(a, rot, norm, grid, s);
}

tp_status run_qk_norm_rope_bwd(const uint16_t* dQKV, const uint16_t* QKV, int64_t N, int n_heads, int n_kv, int head_dim,
                               int t, const QkNormRope& o, uint16_t* out, float* dq_gamma, float* dk_gamma,
                               int accumulate, void* ws, size_t ws_bytes, cudaStream_t s) {
  QkArgs a{};
  int rot;
  bool norm;
  TP_RETURN_IF(check_bwd(dQKV, QKV, N, n_heads, n_kv, head_dim, t, o, out, dq_gamma, dk_gamma, ws, ws_bytes, a, rot,
                         norm));
  TP_RETURN_IF(ready());
  if (N == 0) {
    if (!accumulate) {
      if (dq_gamma) TP_CUDA_CHECK(cudaMemsetAsync(dq_gamma, 0, HD * sizeof(float), s));
      if (dk_gamma) TP_CUDA_CHECK(cudaMemsetAsync(dk_gamma, 0, HD * sizeof(float), s));
    }
    return TP_OK;
  }
  if (dQKV == out) a.nh = a.q_t + a.kv_t;  // in place: dV stays as it is
  a.x = QKV;
  a.dy = dQKV;
  a.y = out;
  a.part = static_cast<float*>(ws);
  a.err = device_error_word();
  a.timeout_ns = wait_timeout_ns();
  unsigned grid = 0;
  const bool bf16 = (o.flags & TP_QKNR_BF16_INPUT) != 0;
  if (o.flags & TP_QKNR_F16_GRAD)
    TP_RETURN_IF((bf16 ? launch_rows<true, true, false>(a, rot, norm, &grid, s)
                       : launch_rows<true, false, false>(a, rot, norm, &grid, s)));
  else
    TP_RETURN_IF((bf16 ? launch_rows<true, true, true>(a, rot, norm, &grid, s)
                       : launch_rows<true, false, true>(a, rot, norm, &grid, s)));
  if (norm && (dq_gamma || dk_gamma)) {
    TP_CUDA_CHECK(launch_pdl(dgamma_final_kernel, dim3(2 * HD / FIN_COLS), dim3(FIN_COLS * FIN_ROWS), 0, s,
                             static_cast<const float*>(a.part), static_cast<int>(grid), dq_gamma, dk_gamma, accumulate));
    count_launch();
  }
  return TP_OK;
}

}  // namespace tp
