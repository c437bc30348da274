"""Thin PyTorch-facing layer over the C ABI: torch allocates device memory and
provides the stream; every step of the TP block runs in libtpshard.so.

The f / g operators of "Tensor and sequence parallelism" (section "How
Megatron partitions") are not separate calls here: with the t ranks resident
on one GPU, f's backward all-reduce and g's forward all-reduce are fixed-order
reductions fused into the row-parallel GEMMs, and the identities are just the
same buffer read by every shard.  :class:`TPMLPFunction` exposes the block as
one autograd Function whose forward is "f, column-parallel, act,
row-parallel, g" and whose backward is the mirror image.
"""

from __future__ import annotations

import ctypes
import functools

import torch

from . import _lib as L

BF16 = torch.bfloat16


def _act(act):
    return L.ACT_BY_NAME[act] if isinstance(act, str) else int(act)


def _ws(nbytes, device):
    return torch.empty(max(int(nbytes), 16), dtype=torch.uint8, device=device)


class MLPWeights:
    """Packed per-shard weights of one TP MLP: W_up (h, F) -> [t][F/t][h],
    W_down (F, h) -> [t][h][F/t]; biases stay as given (b_up is split by the
    same contiguous column blocks)."""

    def __init__(self, W_up, b_up, W_down, b_down, t):
        h, F = W_up.shape
        assert W_down.shape == (F, h) and F % t == 0
        self.h, self.F, self.t = h, F, t
        self.Wup_p = torch.empty(t, F // t, h, dtype=BF16, device=W_up.device)
        self.Wdown_p = torch.empty(t, h, F // t, dtype=BF16, device=W_up.device)
        L.tp_pack_col(W_up, h, F, t, self.Wup_p)
        L.tp_pack_row(W_down, F, h, t, self.Wdown_p)
        self.b_up, self.b_down = b_up, b_down


class SwiGLUWeights(MLPWeights):
    """Packed per-shard weights of a SwiGLU MLP: W_gate and W_up (h, F) -> one
    [t][2F/t][h] block (tp_pack_swiglu: gate and up rows alternate in groups of
    128), W_down (F, h) -> [t][h][F/t].  No biases on the gate / up side."""

    def __init__(self, W_gate, W_up, W_down, b_down, t):
        h, F = W_up.shape
        assert W_gate.shape == (h, F) and W_down.shape == (F, h) and F % t == 0
        self.h, self.F, self.t = h, F, t
        self.Wup_p = torch.empty(t, 2 * F // t, h, dtype=BF16, device=W_up.device)
        self.Wdown_p = torch.empty(t, h, F // t, dtype=BF16, device=W_up.device)
        L.tp_pack_swiglu(W_gate, W_up, h, F, t, self.Wup_p)
        L.tp_pack_row(W_down, F, h, t, self.Wdown_p)
        self.b_up, self.b_down = None, b_down


def _z_cols(w, act):
    """Columns of a shard's Z / dZ: twice F/t under SwiGLU (gate and up)."""
    return (2 if _act(act) == L.ACT_BY_NAME["swiglu"] else 1) * (w.F // w.t)


def mlp_forward(X, w: MLPWeights, act="gelu_tanh", residual=None, save_z=True, flags=0):
    """Y = sum_i act(X W_up,i + b_up,i) W_down,i + b_down (+ residual).  Returns (Y, Z, A).
    With act="swiglu" (SwiGLUWeights) A_i = silu(X W_gate,i) * (X W_up,i) and Z holds
    the gate and up pre-activations, interleaved as in the packed weights."""
    M = X.shape[0]
    Y = torch.empty(M, w.h, dtype=BF16, device=X.device)
    A = torch.empty(w.t, M, w.F // w.t, dtype=BF16, device=X.device)
    swiglu = _act(act) == L.ACT_BY_NAME["swiglu"]
    Z = torch.empty(w.t, M, _z_cols(w, act), dtype=BF16, device=X.device) if (save_z or swiglu) else None
    nws = L.tp_mlp_workspace_size(M, w.h, w.F, w.t, flags)
    ws = _ws(nws, X.device)
    L.tp_mlp_forward(X, M, w.h, w.F, w.t, _act(act), w.Wup_p, w.b_up, w.Wdown_p, w.b_down, residual, Y, Z, A,
                     flags, ws, ws.numel())
    return Y, Z, A


def mlp_backward(dY, X, Z, A, w: MLPWeights, act="gelu_tanh", flags=0, grads=None):
    """Gradients of <Y, dY>.  Returns dict dX, dWup_p, dWdown_p, dbup, dbdown
    (weight grads in the packed layouts, fp32).  Pass `grads` to accumulate."""
    M = X.shape[0]
    acc = grads is not None
    swiglu = _act(act) == L.ACT_BY_NAME["swiglu"]
    if grads is None:
        grads = {"dWup_p": torch.empty(w.t, _z_cols(w, act), w.h, dtype=torch.float32, device=X.device),
                 "dWdown_p": torch.empty(w.t, w.h, w.F // w.t, dtype=torch.float32, device=X.device),
                 "dbup": None if swiglu else torch.empty(w.F, dtype=torch.float32, device=X.device),
                 "dbdown": torch.empty(w.h, dtype=torch.float32, device=X.device)}
    dX = torch.empty(M, w.h, dtype=BF16, device=X.device)
    ws = _ws(L.tp_mlp_backward_workspace_size(M, w.h, w.F, w.t, flags), X.device)
    L.tp_mlp_backward(dY, X, Z, A, M, w.h, w.F, w.t, _act(act), w.Wup_p, w.Wdown_p, dX, grads["dWup_p"],
                      grads["dWdown_p"], grads["dbup"], grads["dbdown"], int(acc), flags, ws, ws.numel())
    out = dict(grads)
    out["dX"] = dX
    return out


class TPMLPFunction(torch.autograd.Function):
    """Autograd wrapper: forward = f (identity) -> column-parallel -> act ->
    row-parallel -> g (fused reduction, bias once); backward = g (identity) ->
    per-shard dgrad / wgrad -> f (fused reduction of the partial dX).
    Weight gradients land in ``weights.grads`` (packed, fp32, accumulated)."""

    @staticmethod
    def forward(ctx, X, weights: MLPWeights, act):
        Y, Z, A = mlp_forward(X.contiguous(), weights, act)
        ctx.save_for_backward(X, Z, A)
        ctx.weights, ctx.act = weights, act
        return Y

    @staticmethod
    def backward(ctx, dY):
        X, Z, A = ctx.saved_tensors
        w = ctx.weights
        prev = getattr(w, "grads", None)
        g = mlp_backward(dY.contiguous(), X, Z, A, w, ctx.act, grads=prev)
        w.grads = {k: g[k] for k in ("dWup_p", "dWdown_p", "dbup", "dbdown")}
        return g["dX"], None, None


# --------------------------------------------------------------------------
# One pre-LN transformer layer: X1 = X + Attn(LN1(X)); Y = X1 + MLP(LN2(X1)).
# With sp=True the LayerNorms and residual adds run on t sequence shards
# ([t][s/t][h], the same bytes as [s][h], so the all-gather entering each TP
# region and the reduce-scatter leaving it are zero-copy) and the LayerNorm
# weight gradients are summed over the shards ("Tensor and sequence
# parallelism", section "Sequence parallelism").  Without SP the LayerNorms are
# replicated: on one GPU that is one LayerNorm over all rows.
# --------------------------------------------------------------------------

class LayerWeights:
    """Packed per-shard weights of one layer (device).  W_qkv is kept in IEEE fp16: the
    layer runs its attention block on an fp16 input (TP_ATTN_F16_INPUT), which the
    softmax of a wide model needs to stay within tolerance."""

    def __init__(self, p, n_heads, head_dim, t):
        d = p["W_qkv"].shape[0]
        F = p["W_up"].shape[1]
        dev = p["W_qkv"].device
        self.d, self.F, self.t, self.n_heads, self.head_dim = d, F, t, n_heads, head_dim
        self.Wqkv_p = torch.empty(t, 3 * d // t, d, dtype=BF16, device=dev)
        self.bqkv_p = torch.empty(t, 3 * d // t, dtype=BF16, device=dev)
        self.Wo_p = torch.empty(t, d, d // t, dtype=BF16, device=dev)
        L.tp_pack_qkv_heads(p["W_qkv"], d, n_heads, head_dim, t, self.Wqkv_p)
        wq16 = torch.empty(t, 3 * d // t, d, dtype=torch.float16, device=dev)
        L.tp_convert_bf16_to_f16(self.Wqkv_p, self.Wqkv_p.numel(), wq16)
        self.Wqkv_p = wq16
        L.tp_pack_qkv_bias(p["b_qkv"], d, n_heads, head_dim, t, self.bqkv_p)
        L.tp_pack_row(p["W_o"], d, d, t, self.Wo_p)
        self.mlp = MLPWeights(p["W_up"], p["b_up"], p["W_down"], p["b_down"], t)
        self.b_o = p["b_o"]
        self.ln1_g, self.ln1_b, self.ln2_g, self.ln2_b = p["ln1_g"], p["ln1_b"], p["ln2_g"], p["ln2_b"]


def layer_forward(X, w: LayerWeights, act="gelu_tanh", causal=True, scale=None, eps=1e-5, sp=False, attn=None):
    """Returns (Y, saved).  X: [s][h] bf16 ([t][s/t][h] when sp).  attn: AttentionOptions (head norms, rotary
    embedding, sliding window with sinks, packed sequences; causal)."""
    s = X.shape[0] if X.dim() == 2 else X.shape[0] * X.shape[1]
    X = X.reshape(s, w.d)
    d, t, dev = w.d, w.t, X.device
    t_ln = t if sp else 1
    scale = (1.0 / w.head_dim ** 0.5) if scale is None else scale
    f32 = torch.float32
    # the attention block's input in IEEE fp16 (TP_ATTN_F16_INPUT)
    Xn1 = torch.empty(s, d, dtype=torch.float16, device=dev)
    m1 = torch.empty(s, dtype=f32, device=dev)
    r1 = torch.empty(s, dtype=f32, device=dev)
    L.tp_sp_layernorm_forward_f16(X, s, d, t_ln, w.ln1_g, w.ln1_b, eps, Xn1, m1, r1)
    X1 = torch.empty(s, d, dtype=BF16, device=dev)
    QKV = torch.empty(t, s, 3 * d // t, dtype=torch.float16, device=dev)  # fp16 attention operands
    O = torch.empty(t, s, d // t, dtype=BF16, device=dev)
    lse = torch.empty(t, w.n_heads // t, s, dtype=f32, device=dev)
    aws = _ws(L.tp_attn_forward_workspace_size(s, d, w.n_heads, w.head_dim, t, 0), dev)  # room for the split-K partials
    QKV_raw = None
    if attn is None:
        L.tp_attn_forward(Xn1, s, d, w.n_heads, w.head_dim, t, int(causal), scale, w.Wqkv_p, w.bqkv_p, w.Wo_p, w.b_o,
                          X, X1, QKV, O, lse, L.TP_ATTN_F16_INPUT, aws, aws.numel())
    else:
        _check(causal, "attention options need causal attention")
        QKV_raw = attn_opt_forward(Xn1, w.Wqkv_p, w.bqkv_p, w.Wo_p, w.b_o, w.n_heads, w.n_heads, t, attn, scale, X,
                                   out=(X1, QKV, O, lse))[1]
    Xn2 = torch.empty(s, d, dtype=BF16, device=dev)
    m2 = torch.empty(s, dtype=f32, device=dev)
    r2 = torch.empty(s, dtype=f32, device=dev)
    L.tp_sp_layernorm_forward(X1, s, d, t_ln, w.ln2_g, w.ln2_b, eps, Xn2, m2, r2)
    Y, Z, A = mlp_forward(Xn2, w.mlp, act, residual=X1)
    saved = dict(X=X, Xn1=Xn1, m1=m1, r1=r1, X1=X1, QKV=QKV, O=O, lse=lse, Xn2=Xn2, m2=m2, r2=r2, Z=Z, A=A,
                 QKV_raw=QKV_raw, attn=attn, s=s, scale=scale, causal=causal, act=act, t_ln=t_ln)
    return Y, saved


def layer_backward(G, saved, w: LayerWeights):
    """Gradients of <Y, G>: dict with dX and every parameter gradient (packed, fp32)."""
    s, d, t, dev = saved["s"], w.d, w.t, G.device
    G = G.reshape(s, d)
    f32 = torch.float32
    g = mlp_backward(G, saved["Xn2"], saved["Z"], saved["A"], w.mlp, saved["act"])
    t_ln = saved["t_ln"]
    dX1 = torch.empty(s, d, dtype=BF16, device=dev)
    ln2 = {k: torch.empty(*shape, dtype=f32, device=dev) for k, shape in
           (("gp", (t_ln, d)), ("bp", (t_ln, d)), ("g", (d,)), ("b", (d,)))}
    L.tp_sp_layernorm_backward(g["dX"], saved["X1"], w.ln2_g, saved["m2"], saved["r2"], G, s, d, t_ln, dX1,
                               ln2["gp"], ln2["bp"], ln2["g"], ln2["b"])
    dXn1 = torch.empty(s, d, dtype=BF16, device=dev)
    dWqkv = torch.empty(t, 3 * d // t, d, dtype=f32, device=dev)
    dbqkv = torch.empty(t, 3 * d // t, dtype=f32, device=dev)
    dWo = torch.empty(t, d, d // t, dtype=f32, device=dev)
    dbo = torch.empty(d, dtype=f32, device=dev)
    head_grads = {}
    if saved["attn"] is None:
        nws = L.tp_attn_backward_workspace_size(s, d, w.n_heads, w.head_dim, t, 0)
        ws = _ws(nws, dev)
        L.tp_attn_backward(dX1, saved["Xn1"], saved["QKV"], saved["O"], saved["lse"], s, d, w.n_heads, w.head_dim, t,
                           int(saved["causal"]), saved["scale"], w.Wqkv_p, w.Wo_p, dXn1, dWqkv, dbqkv, dWo, dbo, 0,
                           L.TP_ATTN_F16_INPUT, ws, nws)
    else:
        g2 = attn_opt_backward(dX1, saved["Xn1"], saved["QKV_raw"], saved["QKV"], saved["O"], saved["lse"], w.Wqkv_p,
                               w.Wo_p, w.n_heads, w.n_heads, t, saved["attn"], saved["scale"],
                               out=(dXn1, dWqkv, dbqkv, dWo, dbo))
        head_grads = {k: g2[k] for k in ("q_gamma", "k_gamma")}
    dX = torch.empty(s, d, dtype=BF16, device=dev)
    ln1 = {k: torch.empty(*shape, dtype=f32, device=dev) for k, shape in
           (("gp", (t_ln, d)), ("bp", (t_ln, d)), ("g", (d,)), ("b", (d,)))}
    L.tp_sp_layernorm_backward(dXn1, saved["X"], w.ln1_g, saved["m1"], saved["r1"], dX1, s, d, t_ln, dX,
                               ln1["gp"], ln1["bp"], ln1["g"], ln1["b"])
    return {**head_grads,
            "dX": dX, "dX1": dX1, "ln1_g": ln1["g"], "ln1_b": ln1["b"], "ln2_g": ln2["g"], "ln2_b": ln2["b"],
            "ln1_g_part": ln1["gp"], "ln2_g_part": ln2["gp"],
            "Wqkv_p": dWqkv, "bqkv_p": dbqkv, "Wo_p": dWo, "b_o": dbo,
            "Wup_p": g["dWup_p"], "b_up": g["dbup"], "Wdown_p": g["dWdown_p"], "b_down": g["dbdown"]}


class DecodeAttnWeights:
    """Packed weights of a TP attention block with grouped-query heads, for
    decode: W_qkv (d, (n_heads + 2 n_kv) head_dim) -> [t][R][d] sharded by KV
    group (replicated KV heads when n_kv < t); W_o (n_heads head_dim, d) ->
    [t][d][n_heads head_dim / t]."""

    def __init__(self, W_qkv, b_qkv, W_o, b_o, n_heads, n_kv, head_dim, t):
        d = W_qkv.shape[0]
        self.d, self.n_heads, self.n_kv, self.head_dim, self.t = d, n_heads, n_kv, head_dim, t
        self.kv_t = n_kv // t if n_kv >= t else 1
        R = (n_heads // t + 2 * self.kv_t) * head_dim
        dev = W_qkv.device
        self.Wqkv_p = torch.empty(t, R, d, dtype=BF16, device=dev)
        L.tp_pack_qkv_gqa(W_qkv, d, n_heads, n_kv, head_dim, t, self.Wqkv_p)
        self.bqkv_p = None
        if b_qkv is not None:
            self.bqkv_p = torch.empty(t, R, dtype=BF16, device=dev)
            L.tp_pack_qkv_gqa_bias(b_qkv, n_heads, n_kv, head_dim, t, self.bqkv_p)
        nq = n_heads * head_dim
        self.Wo_p = torch.empty(t, d, nq // t, dtype=BF16, device=dev)
        L.tp_pack_row(W_o, nq, d, t, self.Wo_p)
        self.b_o = b_o

    def cache_shape(self, B, L_max):
        """Per-shard KV cache [t][kv_t][B][L_max][head_dim] (fp16)."""
        return (self.t, self.kv_t, B, L_max, self.head_dim)

    def workspace(self, B, L_max, device):
        return _ws(L.tp_decode_attn_workspace_size(B, self.d, self.n_heads, self.n_kv, self.head_dim, self.t, L_max),
                   device)


def decode_attn_forward(x, w: DecodeAttnWeights, K_cache, V_cache, pos, scale=None, ws=None, out=None, attn=None):
    """One decode step: appends each sequence's new key/value at pos[b] in
    every shard's cache copy and returns y [B][d] = sum_i O_i W_o,i + b_o.
    Allocates nothing when ws and out are given (so it can be captured in a
    CUDA graph).  attn: AttentionOptions (head norms, rotary embedding, sliding
    window with sinks, rolling caches); pos[b] = -1 then marks an empty row of a
    padded batch; ws: decode_attn_opt_workspace()."""
    B = x.shape[0]
    L_max = K_cache.shape[3]
    assert K_cache.dtype == torch.float16 and V_cache.dtype == torch.float16 and pos.dtype == torch.int32
    if scale is None:
        scale = w.head_dim ** -0.5
    if attn is not None:
        return _decode_attn_opt(x, w, K_cache, V_cache, pos, scale, ws, out, attn)
    if ws is None:
        ws = w.workspace(B, L_max, x.device)
    y = out if out is not None else torch.empty(B, w.d, dtype=BF16, device=x.device)
    L.tp_decode_attn_forward(x, B, w.d, w.n_heads, w.n_kv, w.head_dim, w.t, scale, w.Wqkv_p, w.bqkv_p, w.Wo_p,
                             w.b_o, K_cache, V_cache, L_max, pos, y, ws, ws.numel())
    return y


# --------------------------------------------------------------------------
# Long-context attention: query / key norm with the rotary embedding, and
# attention over a sliding window with sink tokens.  A shard's QKV row is
# [its query heads | its K heads | its V heads], 128 columns a head, as in the
# attention blocks above; n_kv < t replicates KV heads.
# --------------------------------------------------------------------------

HEAD_DIM = 128
_HEAD = (HEAD_DIM,)


def _check(cond, what):
    if not cond:
        raise ValueError(what)


def _tensor(x, name, dtypes, shape, device, optional=False):
    """Checks one tensor argument: dtype, shape, contiguity, device.  (A decode step's kernels take a
    few microseconds, as long as formatting these messages for every call would.)"""
    if x is None:
        _check(optional, name + " is required")
        return
    if x.dtype is dtypes and x.shape == shape and x.device == device and x.is_contiguous():
        return
    if x.dtype is not dtypes and not (type(dtypes) is tuple and x.dtype in dtypes):
        raise ValueError(f"{name}: dtype {x.dtype}, expected {dtypes}")
    if x.shape != shape:
        raise ValueError(f"{name}: shape {tuple(x.shape)}, expected {tuple(shape)}")
    if not x.is_contiguous():
        raise ValueError(name + " must be contiguous")
    if x.device != device:
        raise ValueError(f"{name} is on {x.device}, expected {device}")


def _buffers(out, device, *expected, optional=()):
    """Checks a tuple of output buffers, each (name, dtype, shape) of those expected."""
    if len(out) != len(expected):
        raise ValueError(f"out: {len(out)} buffers, expected {', '.join(name for name, _, _ in expected)}")
    for x, (name, dtype, shape) in zip(out, expected):
        _tensor(x, name + " of out", dtype, shape, device, name in optional)


def _on(device, call, *args):
    """call(*args) with `device` current, on its current stream."""
    if torch._C._cuda_getDevice() == device.index:
        return call(*args)
    with torch.cuda.device(device):
        return call(*args)


def _sizes(entry):
    """A workspace query by its arguments: at least 16 bytes, asked once for each."""
    return functools.lru_cache(maxsize=1024)(lambda *shape: max(int(getattr(L, entry)(*shape)), 16))


_decode_ws_bytes = _sizes("tp_window_decode_workspace_size")
_window_fwd_ws_bytes = _sizes("tp_attn_window_forward_workspace_size")
_window_bwd_ws_bytes = _sizes("tp_attn_window_backward_workspace_size")
_norm_rope_ws_bytes = _sizes("tp_qk_norm_rope_backward_workspace_size")
F16 = torch.float16


def _heads_of(t, R, n_heads, n_kv):
    """KV heads of a shard; checks that rows of width R hold the heads."""
    if not (n_heads >= 1 and n_kv >= 1 and n_heads % t == 0 and n_heads % n_kv == 0 and
            (n_kv % t == 0 if n_kv >= t else t % n_kv == 0)):
        raise ValueError(f"{n_heads} / {n_kv} heads do not split over {t} shards")
    kv_t = n_kv // t if n_kv >= t else 1
    if R != (n_heads // t + 2 * kv_t) * HEAD_DIM:
        raise ValueError(f"row width {R} does not hold {n_heads} / {n_kv} heads of 128 columns on {t} shards")
    return kv_t


def _caches(K, V, t, kv_t, B, dev):
    """Checks the K and V caches [t][kv_t][B][L_max][128]."""
    shape = K.shape
    if not (len(shape) == 5 and shape[:3] == (t, kv_t, B) and shape[4] == HEAD_DIM and V.shape == shape and
            K.dtype is F16 and V.dtype is F16 and K.device == dev and V.device == dev and K.is_contiguous() and
            V.is_contiguous()):
        _check(K.dim() == 5, "K_cache must be [t][kv_t][B][L_max][128]")
        for name, c in (("K_cache", K), ("V_cache", V)):
            _tensor(c, name, F16, (t, kv_t, B, K.shape[3], HEAD_DIM), dev)


def rope_frequencies(rot_dim=HEAD_DIM, base=10000.0, device="cuda"):
    """f_i = base^(-2 i / rot_dim), i < rot_dim / 2, in radians per position: the inv_freq of the
    calls below (any other float64 [rot_dim / 2] tensor, e.g. rescaled frequencies, works too)."""
    i = torch.arange(rot_dim // 2, dtype=torch.float64)
    return (float(base) ** (-2.0 * i / rot_dim)).to(device)


def _norm_rope_args(QKV, n_heads, n_kv, q_gamma, k_gamma, inv_freq, pos, interleaved):
    """Checks what the norm + rotation calls share.  The conditions are written out in one expression (and
    only on a failure once more, to name the argument): they are most of a decode step's host time."""
    shape, dtype, dev = QKV.shape, QKV.dtype, QKV.device
    if len(shape) != 3:
        raise ValueError("QKV must be [t][rows][R]")
    t, N, R = shape
    kv_t = _heads_of(t, R, n_heads, n_kv)
    rot = 0 if inv_freq is None else 2 * inv_freq.numel()
    if not ((dtype is BF16 or dtype is F16) and QKV.is_contiguous() and
            (q_gamma is None if k_gamma is None else
             q_gamma is not None and q_gamma.dtype is BF16 and k_gamma.dtype is BF16 and q_gamma.shape == _HEAD and
             k_gamma.shape == _HEAD and q_gamma.device == dev and k_gamma.device == dev and q_gamma.is_contiguous() and
             k_gamma.is_contiguous()) and
            (q_gamma is not None if inv_freq is None else
             16 <= rot <= HEAD_DIM and rot % 16 == 0 and inv_freq.dtype is torch.float64 and inv_freq.dim() == 1 and
             inv_freq.device == dev and inv_freq.is_contiguous()) and
            (pos is None or (pos.dtype is torch.int32 and pos.shape == (N,) and pos.device == dev and
                             pos.is_contiguous()))):
        _tensor(QKV, "QKV", (F16, BF16), shape, dev)
        _check((q_gamma is None) == (k_gamma is None), "q_gamma and k_gamma go together")
        _tensor(q_gamma, "q_gamma", BF16, _HEAD, dev, True)
        _tensor(k_gamma, "k_gamma", BF16, _HEAD, dev, True)
        _check(q_gamma is not None or inv_freq is not None, "neither a norm nor a rotation")
        _check(inv_freq is None or (16 <= rot <= HEAD_DIM and rot % 16 == 0),
               "rotary dimension: a multiple of 16, 16..128")
        _tensor(inv_freq, "inv_freq", torch.float64, (rot // 2,), dev, True)
        _tensor(pos, "pos", torch.int32, (N,), dev, True)
    flags = (L.TP_QKNR_BF16_INPUT if dtype is BF16 else 0) | (L.TP_ROPE_INTERLEAVED if interleaved else 0)
    return t, N, R, kv_t, rot, flags, dev


def qk_norm_rope_forward(QKV, n_heads, n_kv, q_gamma=None, k_gamma=None, eps=1e-6, inv_freq=None, pos=None,
                         interleaved=False, out=None):
    """RMS norm of every query and key head (q_gamma, k_gamma; left out when None) and the rotary
    embedding (inv_freq; left out when None) of QKV [t][N][R], fp16 or bf16, in one pass.  Returns
    QKV [t][N][R] fp16 with the values carried over; out may be QKV itself (fp16: the values are
    then not touched).  pos: int32 [N], default 0..N-1."""
    t, N, R, _, rot, flags, dev = _norm_rope_args(QKV, n_heads, n_kv, q_gamma, k_gamma, inv_freq, pos, interleaved)
    if out is None:
        out = torch.empty(t, N, R, dtype=F16, device=dev)
    else:
        _tensor(out, "out", F16, QKV.shape, dev)
    _on(dev, L.tp_qk_norm_rope_forward, QKV, N, n_heads, n_kv, HEAD_DIM, t, q_gamma, k_gamma, eps, inv_freq, rot,
        pos, out, flags)
    return out


def qk_norm_rope_backward(dQKV, QKV, n_heads, n_kv, q_gamma=None, k_gamma=None, eps=1e-6, inv_freq=None, pos=None,
                          interleaved=False, out=None, grads=None):
    """Backward of qk_norm_rope_forward: dQKV [t][N][R] (bf16 or fp16) is the gradient of its
    result, QKV its input.  Returns (gradient of QKV, dq_gamma, dk_gamma) -- the first in dQKV's
    type (out may be dQKV itself), the others fp32 [128], None without a norm.  grads =
    (dq_gamma, dk_gamma) accumulates into them."""
    t, N, R, _, rot, flags, dev = _norm_rope_args(QKV, n_heads, n_kv, q_gamma, k_gamma, inv_freq, pos, interleaved)
    _tensor(dQKV, "dQKV", (BF16, torch.float16), QKV.shape, dev)
    if out is None:
        out = torch.empty_like(dQKV)
    else:
        _tensor(out, "out", dQKV.dtype, QKV.shape, dev)
    if dQKV.dtype == torch.float16:
        flags |= L.TP_QKNR_F16_GRAD
    dqg = dkg = ws = None
    if q_gamma is not None:
        if grads is None:
            dqg = torch.empty(HEAD_DIM, dtype=torch.float32, device=dev)
            dkg = torch.empty(HEAD_DIM, dtype=torch.float32, device=dev)
        else:
            dqg, dkg = grads
            _tensor(dqg, "dq_gamma", torch.float32, _HEAD, dev)
            _tensor(dkg, "dk_gamma", torch.float32, _HEAD, dev)
        ws = torch.empty(_norm_rope_ws_bytes(), dtype=torch.uint8, device=dev)
    _on(dev, L.tp_qk_norm_rope_backward, dQKV, QKV, N, n_heads, n_kv, HEAD_DIM, t, q_gamma, k_gamma, eps, inv_freq, rot,
        pos, out, dqg, dkg, int(grads is not None), flags, ws, 0 if ws is None else ws.numel())
    return out, dqg, dkg


def qk_norm_rope_append(QKV, n_heads, n_kv, K_cache, V_cache, pos, q_gamma=None, k_gamma=None, eps=1e-6, inv_freq=None,
                        interleaved=False, window=None, n_sink=0, rolling=False, out=None):
    """The decode form: QKV [t][B][R] holds one token per sequence, at position pos[b] (int32, -1
    for an empty row of a padded batch).  Returns the queries [B][n_heads][128] fp16; the keys and
    values go into the caches [t][kv_t][B][L_max][128] fp16 at slot pos[b], or, rolling, at the
    slot of a cache that keeps the first n_sink and the last `window` positions."""
    t, B, _, kv_t, rot, flags, dev = _norm_rope_args(QKV, n_heads, n_kv, q_gamma, k_gamma, inv_freq, pos, interleaved)
    _caches(K_cache, V_cache, t, kv_t, B, dev)
    L_max = K_cache.shape[3]
    _check(pos is not None, "pos is required")
    _check(not rolling or window is not None, "a rolling cache needs a window")
    if out is None:
        out = torch.empty(B, n_heads, HEAD_DIM, dtype=F16, device=dev)
    else:
        _tensor(out, "out", F16, (B, n_heads, HEAD_DIM), dev)
    _on(dev, L.tp_qk_norm_rope_append, QKV, B, n_heads, n_kv, HEAD_DIM, t, q_gamma, k_gamma, eps, inv_freq, rot, pos,
        out, K_cache, V_cache, L_max, window if rolling else 0, n_sink if rolling else 0, int(bool(rolling)), flags)
    return out


def _window_args(QKV, n_heads, n_kv, window, n_sink, scale, cu_seqlens):
    _check(QKV.dim() == 3, "QKV must be [t][N][R]")
    t, N, R = QKV.shape
    _heads_of(t, R, n_heads, n_kv)
    _tensor(QKV, "QKV", torch.float16, QKV.shape, QKV.device)
    _check(window is None or window >= 1, "window: at least 1, or None for no limit")
    _check(n_sink >= 0, "n_sink: at least 0")
    n_seq = 0
    if cu_seqlens is not None:
        _check(cu_seqlens.dim() == 1 and cu_seqlens.numel() >= 2, "cu_seqlens must be [n_seq + 1], n_seq >= 1")
        _tensor(cu_seqlens, "cu_seqlens", torch.int32, cu_seqlens.shape, QKV.device)
        n_seq = cu_seqlens.numel() - 1
    return t, N, R, max(N, 1) if window is None else int(window), HEAD_DIM ** -0.5 if scale is None else scale, n_seq


def window_attn_forward(QKV, n_heads, n_kv, window=None, n_sink=0, scale=None, cu_seqlens=None, out=None, lse=None):
    """Causal attention of QKV [t][N][R] fp16 in which a query sees the last `window` keys (None: no
    limit) and the first n_sink of its sequence.  cu_seqlens: int32 [n_seq + 1] row boundaries of
    packed sequences; rows behind the last keep what out and lse hold.  Returns (O [t][N][d/t] bf16,
    lse [t][n_heads/t][N] fp32)."""
    t, N, R, window, scale, n_seq = _window_args(QKV, n_heads, n_kv, window, n_sink, scale, cu_seqlens)
    dev = QKV.device
    d, q_t = n_heads * HEAD_DIM, n_heads // t
    if out is None:
        out = torch.empty(t, N, q_t * HEAD_DIM, dtype=BF16, device=dev)
    else:
        _tensor(out, "out", BF16, (t, N, q_t * HEAD_DIM), dev)
    if lse is None:
        lse = torch.empty(t, q_t, N, dtype=torch.float32, device=dev)
    else:
        _tensor(lse, "lse", torch.float32, (t, q_t, N), dev)
    ws = torch.empty(_window_fwd_ws_bytes(N, n_seq), dtype=torch.uint8, device=dev) if n_seq else None
    _on(dev, L.tp_attn_window_forward, QKV, N, d, n_heads, n_kv, HEAD_DIM, t, window, n_sink, scale, cu_seqlens, n_seq,
        out, lse, ws, 0 if ws is None else ws.numel())
    return out, lse


def window_attn_backward(dO, QKV, O, lse, n_heads, n_kv, window=None, n_sink=0, scale=None, cu_seqlens=None, out=None):
    """Gradient of <O, dO> with respect to QKV, from the forward's inputs and results (dO fp16).
    Returns dQKV [t][N][R]: bf16, or fp16 when such an out is given; 0 in rows of no sequence."""
    t, N, R, window, scale, n_seq = _window_args(QKV, n_heads, n_kv, window, n_sink, scale, cu_seqlens)
    dev = QKV.device
    d, q_t = n_heads * HEAD_DIM, n_heads // t
    _tensor(dO, "dO", torch.float16, (t, N, q_t * HEAD_DIM), dev)
    _tensor(O, "O", BF16, (t, N, q_t * HEAD_DIM), dev)
    _tensor(lse, "lse", torch.float32, (t, q_t, N), dev)
    if out is None:
        out = torch.empty(t, N, R, dtype=BF16, device=dev)
    else:
        _tensor(out, "out", (BF16, F16), (t, N, R), dev)
    ws_bytes = _window_bwd_ws_bytes(N, d, n_heads, n_kv, HEAD_DIM, t, window, n_sink, n_seq)
    ws_bytes = (ws_bytes + 255) & ~255
    ws = torch.empty(ws_bytes + 4 * N * n_heads, dtype=torch.uint8, device=dev)  # and, behind it, D [n_heads][N]
    _on(dev, L.tp_attn_window_backward, QKV, O, dO, lse, N, d, n_heads, n_kv, HEAD_DIM, t, window, n_sink, scale,
        cu_seqlens, n_seq, ws.data_ptr() + ws_bytes, out, L.TP_ATTN_F16_INPUT if out.dtype is F16 else 0, ws, ws_bytes)
    return out


def window_decode_attn(Q, K_cache, V_cache, pos, n_kv, window=None, n_sink=0, scale=None, rolling=False, ws=None,
                       out=None):
    """One decode step: Q [B][n_heads][128] fp16 at positions pos (int32 [B], -1 for an empty row)
    against caches [t][kv_t][B][L_max][128] fp16 that hold the tokens' own keys and values already
    (qk_norm_rope_append).  A token sees the last `window` positions (None: no limit) and the first
    n_sink; rolling: of a cache that keeps only those.  Returns O [B][n_heads][128] bf16.  Allocates
    nothing when ws and out are given."""
    shape, dev = Q.shape, Q.device
    _check(len(shape) == 3 and K_cache.dim() == 5, "Q must be [B][n_heads][128], the caches [t][kv_t][B][L_max][128]")
    B, n_heads, _ = shape
    t, kv_t, _, L_max, _ = K_cache.shape
    if not (Q.dtype is F16 and shape[2] == HEAD_DIM and Q.is_contiguous() and pos.dtype is torch.int32 and
            pos.shape == (B,) and pos.device == dev and pos.is_contiguous()):
        _tensor(Q, "Q", F16, (B, n_heads, HEAD_DIM), dev)
        _tensor(pos, "pos", torch.int32, (B,), dev)
    _heads_of(t, (n_heads // t + 2 * kv_t) * HEAD_DIM, n_heads, n_kv)
    _caches(K_cache, V_cache, t, kv_t, B, dev)
    _check(window is None or window >= 1, "window: at least 1, or None for no limit")
    _check(n_sink >= 0, "n_sink: at least 0")
    _check(not rolling or window is not None, "a rolling cache needs a window")
    if ws is None:
        ws = torch.empty(_decode_ws_bytes(B, n_heads, n_kv, HEAD_DIM, t), dtype=torch.uint8, device=dev)
    elif ws.device != dev:
        raise ValueError(f"ws is on {ws.device}, expected {dev}")
    if out is None:
        out = torch.empty(B, n_heads, HEAD_DIM, dtype=BF16, device=dev)
    else:
        _tensor(out, "out", BF16, (B, n_heads, HEAD_DIM), dev)
    _on(dev, L.tp_window_decode_forward, Q, B, n_heads, n_kv, HEAD_DIM, t, L_max if window is None else window, n_sink,
        int(bool(rolling)), HEAD_DIM ** -0.5 if scale is None else scale, K_cache, V_cache, L_max, pos, out, ws,
        ws.numel())
    return out


class AttentionOptions:
    """What the attention blocks do between their projections beyond causal attention: RMS norm of the
    query and key heads (q_gamma, k_gamma [128] bf16), the rotary embedding (inv_freq, e.g.
    rope_frequencies(); pos: int32 positions of the rows, default 0, 1, ..; interleaved pairs), a sliding
    window with n_sink sink tokens, packed sequences (cu_seqlens), and for decode rolling caches that
    keep only the sinks and the window.  Holds the tensors; one object serves any number of calls."""

    def __init__(self, window=None, n_sink=0, q_gamma=None, k_gamma=None, eps=1e-6, inv_freq=None, pos=None,
                 interleaved=False, cu_seqlens=None, rolling=False):
        _check(window is None or window >= 1, "window: at least 1, or None for no limit")
        _check(n_sink >= 0, "n_sink: at least 0")
        _check((q_gamma is None) == (k_gamma is None), "q_gamma and k_gamma go together")
        _check(not rolling or window is not None, "a rolling cache needs a window")
        first = next((x for x in (q_gamma, inv_freq, pos, cu_seqlens) if x is not None), None)
        dev = None if first is None else first.device
        for name, x, dtype, n in (("q_gamma", q_gamma, BF16, HEAD_DIM), ("k_gamma", k_gamma, BF16, HEAD_DIM),
                                  ("inv_freq", inv_freq, torch.float64, None), ("pos", pos, torch.int32, None),
                                  ("cu_seqlens", cu_seqlens, torch.int32, None)):
            if x is not None:
                _check(x.dim() == 1, name + " must have one dimension")
                _tensor(x, name, dtype, (x.numel() if n is None else n,), dev)
        rot = 0 if inv_freq is None else 2 * inv_freq.numel()
        _check(inv_freq is None or (16 <= rot <= HEAD_DIM and rot % 16 == 0),
               "rotary dimension: a multiple of 16, 16..128")
        _check(cu_seqlens is None or cu_seqlens.numel() >= 2, "cu_seqlens must be [n_seq + 1], n_seq >= 1")
        self.window, self.n_sink, self.eps, self.rolling = window, n_sink, eps, bool(rolling)
        self.q_gamma, self.k_gamma, self.inv_freq = q_gamma, k_gamma, inv_freq
        self.pos, self.cu_seqlens, self.device = pos, cu_seqlens, dev
        ptr = lambda x: None if x is None else x.data_ptr()  # noqa: E731
        n_seq = 0 if cu_seqlens is None else cu_seqlens.numel() - 1
        self._struct = L.AttnOptions(window or 0, n_sink, ptr(cu_seqlens), n_seq, ptr(q_gamma), ptr(k_gamma),
                                     ptr(inv_freq), ptr(pos), eps, rot, L.TP_ROPE_INTERLEAVED if interleaved else 0,
                                     int(self.rolling))
        self.ptr = ctypes.addressof(self._struct)

    def check(self, device, rows=None):
        _check(self.device is None or self.device == device, f"options on {self.device}, expected {device}")
        _check(rows is None or self.pos is None or self.pos.numel() == rows, "pos must have one position a row")


def _block_args(X, Wqkv_p, Wo_p, n_heads, n_kv, t):
    """Checks X [N][d] and the packed weights of a grouped-query attention block."""
    _check(X.dim() == 2, "X must be [N][d]")
    N, d = X.shape
    q_t = n_heads // t
    R = (q_t + 2 * (n_kv // t if n_kv >= t else 1)) * HEAD_DIM
    _heads_of(t, R, n_heads, n_kv)
    _check(d == n_heads * HEAD_DIM and Wqkv_p.shape == (t, R, d), "X and W_qkv do not hold these heads")
    _check(Wqkv_p.dtype == X.dtype, "X and W_qkv have one type")
    _tensor(X, "X", (BF16, F16), (N, d), X.device)
    _tensor(Wqkv_p, "Wqkv_p", X.dtype, (t, R, d), X.device)
    _tensor(Wo_p, "Wo_p", BF16, (t, d, q_t * HEAD_DIM), X.device)
    return N, d, q_t, R


def attn_opt_forward(X, Wqkv_p, bqkv_p, Wo_p, b_o, n_heads, n_kv, t, attn, scale=None, residual=None, keep_raw=True,
                     out=None):
    """The grouped-query attention block (packed weights) with AttentionOptions: X [N][d] bf16, or fp16 with
    W_qkv in fp16.  Returns (Y, QKV_raw, QKV, O, lse); QKV_raw, the projection before norm and rotation, is
    kept for the backward of head norms (keep_raw), else None.  out = (Y, QKV, O, lse) buffers."""
    N, d, q_t, R = _block_args(X, Wqkv_p, Wo_p, n_heads, n_kv, t)
    dev = X.device
    _tensor(bqkv_p, "bqkv_p", BF16, (t, R), dev, True)
    _tensor(b_o, "b_o", BF16, (d,), dev, True)
    _tensor(residual, "residual", BF16, (N, d), dev, True)
    attn.check(dev, N)
    if out is None:
        out = (torch.empty(N, d, dtype=BF16, device=dev), torch.empty(t, N, R, dtype=torch.float16, device=dev),
               torch.empty(t, N, q_t * HEAD_DIM, dtype=BF16, device=dev),
               torch.empty(t, q_t, N, dtype=torch.float32, device=dev))
    else:
        _buffers(out, dev, ("Y", BF16, (N, d)), ("QKV", F16, (t, N, R)), ("O", BF16, (t, N, q_t * HEAD_DIM)),
                 ("lse", torch.float32, (t, q_t, N)))
    Y, QKV, O, lse = out
    raw = torch.empty_like(QKV) if keep_raw and attn.q_gamma is not None else None
    ws = _ws(L.tp_attn_opt_forward_workspace_size(N, d, n_heads, n_kv, HEAD_DIM, t, attn.ptr), dev)
    _on(dev, L.tp_attn_opt_forward, X, N, d, n_heads, n_kv, HEAD_DIM, t, HEAD_DIM ** -0.5 if scale is None else scale,
        attn.ptr, Wqkv_p, bqkv_p, Wo_p, b_o, residual, Y, raw, QKV, O, lse,
        L.TP_ATTN_F16_INPUT if X.dtype == torch.float16 else 0, ws, ws.numel())
    return Y, raw, QKV, O, lse


def attn_opt_backward(dY, X, QKV_raw, QKV, O, lse, Wqkv_p, Wo_p, n_heads, n_kv, t, attn, scale=None, out=None):
    """Gradients of <Y, dY> of attn_opt_forward: dict of dX, Wqkv_p, bqkv_p, Wo_p, b_o, q_gamma, k_gamma
    (parameters fp32, packed; the gammas None without norms).  out = (dX, dWqkv, dbqkv, dWo, dbo) buffers (a
    bias gradient that is None is left out)."""
    N, d, q_t, R = _block_args(X, Wqkv_p, Wo_p, n_heads, n_kv, t)
    dev = X.device
    f32 = dict(dtype=torch.float32, device=dev)
    _tensor(dY, "dY", BF16, (N, d), dev)
    _tensor(QKV_raw, "QKV_raw", F16, (t, N, R), dev, attn.q_gamma is None)
    _tensor(QKV, "QKV", F16, (t, N, R), dev)
    _tensor(O, "O", BF16, (t, N, q_t * HEAD_DIM), dev)
    _tensor(lse, "lse", torch.float32, (t, q_t, N), dev)
    attn.check(dev, N)
    if out is None:
        out = (torch.empty(N, d, dtype=BF16, device=dev), torch.empty(Wqkv_p.shape, **f32),
               torch.empty(Wqkv_p.shape[:2], **f32), torch.empty(Wo_p.shape, **f32), torch.empty(d, **f32))
    else:
        _buffers(out, dev, ("dX", BF16, (N, d)), ("dWqkv", torch.float32, Wqkv_p.shape),
                 ("dbqkv", torch.float32, Wqkv_p.shape[:2]), ("dWo", torch.float32, Wo_p.shape),
                 ("dbo", torch.float32, (d,)), optional=("dbqkv", "dbo"))
    dX, dWqkv, dbqkv, dWo, dbo = out
    dqg = dkg = None
    if attn.q_gamma is not None:
        dqg, dkg = torch.empty(HEAD_DIM, **f32), torch.empty(HEAD_DIM, **f32)
    ws = _ws(L.tp_attn_opt_backward_workspace_size(N, d, n_heads, n_kv, HEAD_DIM, t, attn.ptr), dev)
    _on(dev, L.tp_attn_opt_backward, dY, X, QKV_raw, QKV, O, lse, N, d, n_heads, n_kv, HEAD_DIM, t,
        HEAD_DIM ** -0.5 if scale is None else scale, attn.ptr, Wqkv_p, Wo_p, dX, dWqkv, dbqkv, dWo, dbo, dqg, dkg, 0,
        L.TP_ATTN_F16_INPUT if X.dtype == torch.float16 else 0, ws, ws.numel())
    return dict(dX=dX, Wqkv_p=dWqkv, bqkv_p=dbqkv, Wo_p=dWo, b_o=dbo, q_gamma=dqg, k_gamma=dkg)


def decode_attn_opt_workspace(B, w: DecodeAttnWeights, device):
    """Workspace of decode_attn_forward with AttentionOptions."""
    return _ws(L.tp_decode_attn_opt_workspace_size(B, w.d, w.n_heads, w.n_kv, w.head_dim, w.t), device)


def _decode_attn_opt(x, w, K_cache, V_cache, pos, scale, ws, out, attn):
    B, dev = x.shape[0], x.device
    L_max = K_cache.shape[3]
    for name, c in (("K_cache", K_cache), ("V_cache", V_cache)):
        _tensor(c, name, torch.float16, (w.t, w.kv_t, B, L_max, HEAD_DIM), dev)
    _tensor(x, "x", BF16, (B, w.d), dev)
    _tensor(pos, "pos", torch.int32, (B,), dev)
    attn.check(dev)
    if ws is None:
        ws = decode_attn_opt_workspace(B, w, dev)
    elif ws.device != dev:
        raise ValueError(f"ws is on {ws.device}, expected {dev}")
    if out is None:
        out = torch.empty(B, w.d, dtype=BF16, device=dev)
    else:
        _tensor(out, "out", BF16, (B, w.d), dev)
    _on(dev, L.tp_decode_attn_opt_forward, x, B, w.d, w.n_heads, w.n_kv, w.head_dim, w.t, scale, attn.ptr, w.Wqkv_p,
        w.bqkv_p, w.Wo_p, w.b_o, K_cache, V_cache, L_max, pos, out, ws, ws.numel())
    return out
