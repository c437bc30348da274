"""The attention blocks and the transformer layer with head norms, rotary embedding and window attention
against the fp64 oracle: forward, every gradient, and the decode step."""

import numpy as np
import pytest
import torch

import oracle as O
from gpu_helpers import assert_close, f64
from megatron_tensor_transformer_shard_gb300 import _lib as L
from megatron_tensor_transformer_shard_gb300 import inputs as I
from megatron_tensor_transformer_shard_gb300 import tp as T

pytestmark = pytest.mark.gpu

SCALE = 128 ** -0.5


def options(norm, rot, window, sink, cu=None, pos=None, inter=False, rolling=False, seed=7):
    g = torch.Generator().manual_seed(seed)
    gq, gk = [(1 + 0.2 * torch.randn(128, generator=g)).to(torch.bfloat16) if norm else None for _ in range(2)]
    f = T.rope_frequencies(rot, 10000.0, "cpu") if rot else None
    dev = lambda x, dt=None: None if x is None else torch.as_tensor(x, dtype=dt).cuda()  # noqa: E731
    opt = T.AttentionOptions(window, sink, dev(gq), dev(gk), 1e-5, dev(f), dev(pos, torch.int32), inter,
                             dev(cu, torch.int32), rolling)
    host = dict(gq=None if gq is None else f64(gq), gk=None if gk is None else f64(gk),
                f=None if f is None else f.numpy(), pos=pos, inter=inter, cu=cu, window=window, sink=sink)
    return opt, host


def oracle_block(X, Wq, bq, Wo, bo, n_heads, n_kv, t, o, dY=None):
    """One attention block on packed weights, in fp64; rows of no sequence have O = 0."""
    N = X.shape[0]
    raw = np.stack([X @ Wq[i].T + bq[i] for i in range(t)])
    n = N if o["cu"] is None else o["cu"][-1]
    rope = o["f"] is not None or o["gq"] is not None
    kw = dict(eps=1e-5, inv_freq=o["f"], pos=o["pos"], interleaved=o["inter"])
    QKV = O.qk_norm_rope(raw, n_heads, n_kv, o["gq"], o["gk"], **kw)[0] if rope else raw
    W = N if o["window"] is None else o["window"]
    dO = None
    if dY is not None:
        dO = np.stack([dY @ Wo[i] for i in range(t)])
    a = O.window_attention(QKV, n_heads, n_kv, W, o["sink"], SCALE, o["cu"], dO)
    Oa = a["O"].copy()
    Oa[:, n:] = 0
    Y = sum(Oa[i] @ Wo[i].T for i in range(t)) + bo
    if dY is None:
        return Y
    dQ = a["dQKV"]
    gq = gk = None
    if rope:
        dQ, gq, gk = O.qk_norm_rope_backward(dQ, raw, n_heads, n_kv, o["gq"], o["gk"], **kw)[:3]
        gq, gk = (gq, gk) if o["gq"] is not None else (None, None)
    return dict(Y=Y, dX=sum(dQ[i] @ Wq[i] for i in range(t)), Wqkv_p=np.stack([dQ[i].T @ X for i in range(t)]),
                bqkv_p=dQ.sum(1), Wo_p=np.stack([dY.T @ Oa[i] for i in range(t)]), b_o=dY.sum(0), q_gamma=gq, k_gamma=gk)


CASES = [  # heads, KV heads, t, N, norm, rotary dimension, window, sinks, boundaries, interleaved, fp16 input
    (4, 2, 2, 200, True, 128, 48, 4, None, False, True),
    (8, 2, 2, 333, True, 64, 100, 3, [0, 90, 91, 300], True, False),
    (4, 4, 4, 150, False, 128, None, 0, None, False, True),
    (8, 1, 4, 260, True, 0, 31, 0, [0, 100, 260], False, True),     # norms without rotation, replicated KV heads
    (4, 2, 1, 140, False, 0, 20, 2, None, False, False),            # a window alone
]


@pytest.mark.parametrize("n_heads,n_kv,t,N,norm,rot,window,sink,cu,inter,f16", CASES)
def test_block(n_heads, n_kv, t, N, norm, rot, window, sink, cu, inter, f16):
    d = n_heads * 128
    inp = I.gqa_attn_inputs(N, d, n_heads, n_kv, 128, seed=3)
    pos = (np.arange(N) * 3 + 1000).astype(np.int32) if rot else None
    opt, host = options(norm, rot, window, sink, cu, pos, inter)
    dev = {k: v.cuda() for k, v in inp.items()}
    w = T.DecodeAttnWeights(dev["W_qkv"], dev["b_qkv"], dev["W_o"], dev["b_o"], n_heads, n_kv, 128, t)
    X, Wq = (dev["X"].half(), w.Wqkv_p.half()) if f16 else (dev["X"], w.Wqkv_p)
    ref = oracle_block(f64(X), f64(Wq), f64(w.bqkv_p), f64(w.Wo_p), f64(w.b_o), n_heads, n_kv, t, host, f64(dev["dY"]))
    out = T.attn_opt_forward(X, Wq, w.bqkv_p, w.Wo_p, w.b_o, n_heads, n_kv, t, opt)
    assert_close("Y", f64(out[0]), ref["Y"])
    g = T.attn_opt_backward(dev["dY"], X, *out[1:], Wq, w.Wo_p, n_heads, n_kv, t, opt)
    for k, v in ref.items():
        if k != "Y" and v is not None:
            assert_close(k, f64(g[k]), v)
    if not norm:
        assert g["q_gamma"] is None
    if cu is not None:
        assert not g["dX"][cu[-1]:].any()
    # inference keeps no raw rows and gives the same result
    again = T.attn_opt_forward(X, Wq, w.bqkv_p, w.Wo_p, w.b_o, n_heads, n_kv, t, opt, keep_raw=False)
    assert again[1] is None and torch.equal(again[0], out[0])
    assert L.tp_get_device_status(check=False) == L.TP_OK


@pytest.mark.parametrize("sp", [False, True])
def test_layer(sp):
    N, d, F, t = 256, 512, 1024, 2
    nh = d // 128
    inp = I.layer_inputs(N, d, F, seed=5)
    opt, host = options(True, 128, 70, 4, [0, 60, 256])
    dev = {k: v.cuda() for k, v in inp.items()}
    w = T.LayerWeights(dev, nh, 128, t)
    Y, saved = T.layer_forward(dev["X"], w, sp=sp, attn=opt)
    g = T.layer_backward(dev["dY"], saved, w)
    r = {k: f64(v) for k, v in inp.items()}
    xn1, m1, r1 = O.layernorm_forward(r["X"], r["ln1_g"], r["ln1_b"], 1e-5)
    args = (f64(w.Wqkv_p), f64(w.bqkv_p), f64(w.Wo_p), r["b_o"], nh, nh, t, host)
    X1 = r["X"] + oracle_block(xn1, *args)
    xn2, m2, r2 = O.layernorm_forward(X1, r["ln2_g"], r["ln2_b"], 1e-5)
    mlp = O.mlp_forward_sharded(xn2, r["W_up"], r["b_up"], r["W_down"], r["b_down"], "gelu_tanh", t)
    assert_close("X1", f64(saved["X1"]), X1)
    assert_close("Y", f64(Y), X1 + mlp["Y"])
    bm = O.mlp_backward_sharded(r["dY"], xn2, r["W_up"], r["W_down"], mlp, "gelu_tanh", t)
    dx2, dg2, _ = O.layernorm_backward(bm["dX"], X1, r["ln2_g"], m2, r2)
    dX1 = r["dY"] + dx2
    b = oracle_block(xn1, *args, dY=dX1)
    dx1, dg1, db1 = O.layernorm_backward(b["dX"], r["X"], r["ln1_g"], m1, r1)
    for k, v in dict(dX=dX1 + dx1, ln1_g=dg1, ln1_b=db1, ln2_g=dg2, Wqkv_p=b["Wqkv_p"], bqkv_p=b["bqkv_p"],
                     Wo_p=b["Wo_p"], b_o=b["b_o"], q_gamma=b["q_gamma"], k_gamma=b["k_gamma"]).items():
        assert_close(k, f64(g[k]), v)
    assert L.tp_get_device_status(check=False) == L.TP_OK


@pytest.mark.parametrize("rolling", [False, True])
@pytest.mark.parametrize("B,n_heads,n_kv,t", [(1, 4, 2, 2), (5, 8, 2, 4), (40, 4, 4, 1)])
def test_decode_token_by_token(B, n_heads, n_kv, t, rolling):
    """Every step's y against the block over the whole sequences; rows finish at different steps."""
    d, steps, window, sink = n_heads * 128, 9, 4, 2
    L_max = window + sink if rolling else steps
    rng = np.random.default_rng(0)
    lens = rng.integers(1, steps + 1, B)
    lens[0] = steps
    inp = I.decode_attn_inputs(1, d, n_heads, n_kv, 128, 1, seed=2)
    g = torch.Generator().manual_seed(4)
    X = torch.randn(B, steps, d, generator=g).to(torch.bfloat16)
    opt, host = options(True, 128, window, sink, rolling=rolling)
    dev = {k: v.cuda() for k, v in inp.items()}
    w = T.DecodeAttnWeights(dev["W_qkv"], dev["b_qkv"], dev["W_o"], dev["b_o"], n_heads, n_kv, 128, t)
    ref = np.stack([oracle_block(f64(X[b]), f64(w.Wqkv_p), f64(w.bqkv_p), f64(w.Wo_p), f64(w.b_o), n_heads, n_kv, t, host)
                    for b in range(B)])
    K, V = (torch.full(w.cache_shape(B, L_max), float("nan"), dtype=torch.float16, device="cuda") for _ in range(2))
    ws = T.decode_attn_opt_workspace(B, w, "cuda")
    y = torch.empty(B, d, dtype=torch.bfloat16, device="cuda")
    pos = torch.zeros(B, dtype=torch.int32, device="cuda")
    x = X[:, 0].cuda().contiguous()
    T.decode_attn_forward(x, w, K, V, pos, ws=ws, out=y, attn=opt)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        T.decode_attn_forward(x, w, K, V, pos, ws=ws, out=y, attn=opt)
    for p in range(steps):
        pos.copy_(torch.tensor([p if p < n else -1 for n in lens], dtype=torch.int32))
        x.copy_(X[:, p])
        graph.replay()
        live = np.nonzero(lens > p)[0]
        assert_close(f"y at {p}", f64(y)[live], ref[live, p])
    assert L.tp_get_device_status(check=False) == L.TP_OK


def test_decode_without_options_is_the_plain_decode():
    B, n_heads, n_kv, t, L_max = 3, 8, 2, 2, 200
    inp = I.decode_attn_inputs(B, 1024, n_heads, n_kv, 128, L_max, seed=1)
    dev = {k: v.cuda() for k, v in inp.items()}
    w = T.DecodeAttnWeights(dev["W_qkv"], dev["b_qkv"], dev["W_o"], dev["b_o"], n_heads, n_kv, 128, t)
    K = dev["K"].view(w.cache_shape(B, L_max)).clone()
    V = dev["V"].view(w.cache_shape(B, L_max)).clone()
    pos = torch.tensor([199, 0, 77], dtype=torch.int32, device="cuda")
    y = T.decode_attn_forward(dev["x"], w, K.clone(), V.clone(), pos)
    y2 = T.decode_attn_forward(dev["x"], w, K, V, pos, attn=T.AttentionOptions())
    assert_close("y", f64(y2), f64(y))


@pytest.mark.parametrize("B,n_heads,n_kv,t,L_max", [(1, 8, 2, 2, 16384), (8, 8, 2, 2, 4096), (40, 4, 4, 1, 300)])
def test_decode_without_options_gives_the_bits_of_the_plain_decode(B, n_heads, n_kv, t, L_max):
    """The same projection, rounded once to fp16, and as many tiles as CTAs or more on both sides, so the same cut."""
    inp = I.decode_attn_inputs(B, n_heads * 128, n_heads, n_kv, 128, L_max, seed=1)
    dev = {k: v.cuda() for k, v in inp.items()}
    w = T.DecodeAttnWeights(dev["W_qkv"], dev["b_qkv"], dev["W_o"], dev["b_o"], n_heads, n_kv, 128, t)
    K, V = (dev[c].view(w.cache_shape(B, L_max)) for c in "KV")
    pos = torch.randint(0, L_max, (B,), generator=torch.Generator().manual_seed(2)).to(torch.int32).cuda()
    pos[0] = L_max - 1
    K1, V1, K2, V2 = K.clone(), V.clone(), K.clone(), V.clone()
    y = T.decode_attn_forward(dev["x"], w, K1, V1, pos)
    y2 = T.decode_attn_forward(dev["x"], w, K2, V2, pos, attn=T.AttentionOptions())
    assert torch.equal(K2, K1) and torch.equal(V2, V1) and torch.equal(y2, y)
    assert not torch.equal(K1, K)


@pytest.mark.parametrize("B", [1, 5, 40])
def test_decode_holds_its_rows_in_fp16(B):
    """The cached value is the projection rounded once to fp16, with norms and rotation on: half a step, and an
    fp32 sum of 512 products (512 half steps of fp32 on the sum of absolute values at most)."""
    n_heads, n_kv, t = 4, 2, 2
    inp = I.decode_attn_inputs(B, 512, n_heads, n_kv, 128, 4, seed=3)
    dev = {k: v.cuda() for k, v in inp.items()}
    w = T.DecodeAttnWeights(dev["W_qkv"], dev["b_qkv"], dev["W_o"], dev["b_o"], n_heads, n_kv, 128, t)
    opt, host = options(True, 128, 4, 1)
    K, V = (torch.zeros(w.cache_shape(B, 4), dtype=torch.float16, device="cuda") for _ in range(2))
    T.decode_attn_forward(dev["x"], w, K, V, torch.zeros(B, dtype=torch.int32, device="cuda"), attn=opt)
    x, Wq, bq = f64(inp["x"]), f64(w.Wqkv_p), f64(w.bqkv_p)
    for i in range(t):
        rows, mag = x @ Wq[i].T + bq[i], np.abs(x) @ np.abs(Wq[i]).T + np.abs(bq[i])
        got, ref = f64(V[i, 0, :, 0]), rows[:, -128:]
        assert (np.abs(got - ref) <= 2.0 ** -11 * np.abs(ref) + 512 * 2.0 ** -24 * mag[:, -128:] + 2.0 ** -25).all()
        # position 0 is not rotated: the normed key, whose roundings the oracle's tolerance counts, of a row off by
        # as much as the value (twice: the norm's factor)
        key, tol = O.qk_norm_rope(rows[None], n_heads // t, 1, host["gq"], host["gk"], 1e-5)
        part, gain = slice(256, 384), np.abs(host["gk"]) / np.sqrt((rows[:, 256:384] ** 2).mean(1, keepdims=True))
        off = 2.0 ** -11 * np.abs(rows[:, part]) + 512 * 2.0 ** -24 * mag[:, part] + 2.0 ** -25
        off = (off + np.abs(rows[:, part]) * (off ** 2).mean(1, keepdims=True) ** 0.5 /
               np.sqrt((rows[:, part] ** 2).mean(1, keepdims=True))) * gain
        assert (np.abs(f64(K[i, 0, :, 0]) - key[0][:, part]) <= tol[0][:, part] + off).all()


def test_padding_of_zeros_leaves_the_gradients_alone():
    """Rows of no sequence that are zeros, no bias, eps = 0: their norm has nothing to divide by, and the parameters'
    gradients are those of the sequences alone."""
    n_heads, n_kv, t, N, n = 4, 2, 2, 200, 130
    inp = I.gqa_attn_inputs(N, 512, n_heads, n_kv, 128, bias=False, seed=3)
    dev = {k: v.cuda() for k, v in inp.items() if v is not None}
    w = T.DecodeAttnWeights(dev["W_qkv"], None, dev["W_o"], None, n_heads, n_kv, 128, t)
    g = torch.ones(128, dtype=torch.bfloat16, device="cuda")
    cu = torch.tensor([0, 60, n], dtype=torch.int32, device="cuda")
    X, dY = dev["X"].clone(), dev["dY"].clone()
    X[n:], dY[n:] = 0, 0

    def grads(X, dY, cu):
        opt = T.AttentionOptions(50, 2, g, g, 0.0, T.rope_frequencies(128), cu_seqlens=cu)
        out = T.attn_opt_forward(X, w.Wqkv_p, None, w.Wo_p, None, n_heads, n_kv, t, opt)
        return T.attn_opt_backward(dY, X, *out[1:], w.Wqkv_p, w.Wo_p, n_heads, n_kv, t, opt)
    a, b = grads(X, dY, cu), grads(X[:n].contiguous(), dY[:n].contiguous(), cu)
    assert not a["dX"][n:].any()
    for k in ("q_gamma", "k_gamma", "Wqkv_p", "Wo_p"):
        assert torch.isfinite(a[k]).all()
        assert_close(k, f64(a[k]), f64(b[k]), 1e-5)
    assert_close("dX", f64(a["dX"][:n]), f64(b["dX"]))


def test_block_in_a_replayed_graph():
    """Forward and backward of the block captured once, replayed with other rows, positions and boundaries."""
    n_heads, n_kv, t, N = 8, 2, 2, 300
    inp = I.gqa_attn_inputs(N, 1024, n_heads, n_kv, 128, seed=3)
    dev = {k: v.cuda() for k, v in inp.items()}
    w = T.DecodeAttnWeights(dev["W_qkv"], dev["b_qkv"], dev["W_o"], dev["b_o"], n_heads, n_kv, 128, t)
    opt, _ = options(True, 128, 48, 3, [0, 100, 300], np.arange(N))
    X, dY = dev["X"].clone(), dev["dY"].clone()

    def both():
        out = T.attn_opt_forward(X, w.Wqkv_p, w.bqkv_p, w.Wo_p, w.b_o, n_heads, n_kv, t, opt)
        g = T.attn_opt_backward(dY, X, *out[1:], w.Wqkv_p, w.Wo_p, n_heads, n_kv, t, opt)
        return [out[0], *g.values()]
    both()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = both()
    for seed, cu in ((1, [0, 7, 300]), (2, [0, 200, 257]), (3, [0, 0, 1])):
        g = torch.Generator().manual_seed(seed)
        X.copy_(torch.randn(N, 1024, generator=g))
        dY.copy_(2.0 ** -8 * seed * torch.randn(N, 1024, generator=g))
        opt.cu_seqlens.copy_(torch.tensor(cu, dtype=torch.int32))
        opt.pos.add_(1000)
        graph.replay()
        torch.cuda.synchronize()
        kept = [x.clone() for x in got]
        for a, b in zip(kept, both()):
            assert torch.equal(a, b)
    assert L.tp_get_device_status(check=False) == L.TP_OK
