"""Decode attention over a sliding window with sink tokens on the GPU against the fp64 oracle, whole and
rolling caches, and the two decode operators run together against the training-shaped forward."""

import numpy as np
import pytest
import torch

import oracle as O
from gpu_helpers import Guarded, f64, guarded_ws
from megatron_tensor_transformer_shard_gb300 import _lib as L
from megatron_tensor_transformer_shard_gb300 import tp as T

pytestmark = pytest.mark.gpu

SCALE = 128 ** -0.5


def rnd(seed, *shape, std=1.0, dtype=torch.float16):
    g = torch.Generator().manual_seed(seed)
    return (std * torch.randn(*shape, generator=g)).to(dtype)


def within(got, ref, tol):
    got = f64(got)
    bad = ~(np.abs(got - ref) <= tol)
    assert not bad.any(), (f"{bad.sum()} of {bad.size} off, first at {np.argwhere(bad)[0]}: "
                           f"{got[bad][0]} for {ref[bad][0]}, tolerance {tol[bad][0]}")


CASES = [  # (heads, KV heads, t), window, sinks, rolling, cache length, positions, scale
    ((2, 1, 1), 1, 0, False, 1, [0], SCALE),
    ((2, 1, 1), 1, 0, True, 1, [10 ** 6], SCALE),
    ((8, 1, 1), 64, 4, False, 300, [299, 0, 67, 68, 150], SCALE),
    ((8, 1, 1), 64, 4, True, 68, [299, 0, 67, 68, 2 ** 31 - 1], SCALE),
    ((64, 8, 4), 128, 4, False, 513, [512, 131, -1, 132, 127, 128, -1], SCALE),
    ((24, 2, 1), 200, 130, False, 700, [699, 330, 329, 128], SCALE),       # 12 heads a group; sinks over two tiles
    ((32, 1, 1), 100, 0, False, 260, [259, 99, 100], SCALE),               # 32 heads a group
    ((8, 2, 4), 256, 5, True, 300, [255, 260, 261, 5000, -1], SCALE),      # replicated KV heads, slots to spare
    ((4, 4, 2), 10 ** 9, 3, False, 333, [332, 100, 0], SCALE),             # no limit in reach
    ((4, 4, 2), 50, 10 ** 9, False, 333, [332, 100, 0], SCALE),            # every key a sink
    ((4, 2, 1), 33, 1, False, 200, [150, 199], -0.1),
    ((4, 2, 1), 33, 1, False, 200, [150, 199], 1.5),
]


@pytest.mark.parametrize("heads,window,sink,rolling,L_max,pos,scale", CASES)
def test_decode(heads, window, sink, rolling, L_max, pos, scale):
    n_heads, n_kv, t = heads
    kv_t = O.tp_long_context.heads_of(*heads)[1]
    B = len(pos)
    Q, K, V = rnd(1, B, n_heads, 128), rnd(2, t, kv_t, B, L_max, 128), rnd(3, t, kv_t, B, L_max, 128)
    ref, tol = O.window_decode(f64(Q), f64(K), f64(V), pos, window, sink, scale, rolling)
    hidden = torch.ones(B, L_max, dtype=torch.bool)
    for b, p in enumerate(pos):
        if p >= 0:
            hidden[b, O.decode_keys(p, window, sink, rolling)] = False
    K[:, :, hidden], V[:, :, hidden] = float("nan"), float("inf")  # slots that no token sees may hold anything
    out = Guarded((B, n_heads, 128), torch.bfloat16)
    before = out.t.clone()
    ws = guarded_ws(L.tp_window_decode_workspace_size(B, n_heads, n_kv, 128, t))
    args = (Q.cuda(), K.cuda(), V.cuda(), torch.tensor(pos, dtype=torch.int32, device="cuda"), n_kv, window, sink, scale,
            rolling)
    T.window_decode_attn(*args, ws=ws.t, out=out.t)
    out.check("O")
    ws.check("workspace")
    live = [b for b, p in enumerate(pos) if p >= 0]
    dead = [b for b, p in enumerate(pos) if p < 0]
    within(out.t[live], ref[live], tol[live])
    assert torch.equal(out.t[dead].view(torch.int16), before[dead].view(torch.int16))
    assert torch.equal(T.window_decode_attn(*args)[live], out.t[live])
    assert L.tp_get_device_status(check=False) == L.TP_OK


def test_full_batch_of_ragged_lengths():
    heads, window, sink, L_max, B = (16, 2, 2), 300, 4, 1024, 256
    rng = np.random.default_rng(0)
    pos = rng.integers(0, L_max, B).tolist()
    pos[0], pos[17], pos[18], pos[255] = L_max - 1, -1, -1, -1
    Q, K, V = rnd(1, B, 16, 128), rnd(2, 2, 1, B, L_max, 128), rnd(3, 2, 1, B, L_max, 128)
    ref, tol = O.window_decode(f64(Q), f64(K), f64(V), pos, window, sink, SCALE)
    got = T.window_decode_attn(Q.cuda(), K.cuda(), V.cuda(), torch.tensor(pos, dtype=torch.int32, device="cuda"), 2,
                               window, sink)
    live = [b for b, p in enumerate(pos) if p >= 0]
    within(got[live], ref[live], tol[live])


def test_nothing_but_empty_rows():
    out = Guarded((3, 4, 128), torch.bfloat16)
    before = out.t.clone()
    z = torch.zeros(1, 2, 3, 64, 128, dtype=torch.float16, device="cuda")
    pos = torch.full((3,), -1, dtype=torch.int32, device="cuda")
    T.window_decode_attn(rnd(1, 3, 4, 128).cuda(), z, z, pos, 2, 8, out=out.t)
    out.check("O")
    assert torch.equal(out.t.view(torch.int16), before.view(torch.int16))
    assert T.window_decode_attn(z[0, 0, :0, :4], z[:, :, :0], z[:, :, :0], pos[:0], 2, 8).shape == (0, 4, 128)


@pytest.mark.parametrize("bad", [-2, 64, 2 ** 31 - 1])
def test_positions_past_the_cache_are_reported(bad):
    Q, K, V = rnd(1, 2, 4, 128).cuda(), rnd(2, 1, 2, 2, 64, 128).cuda(), rnd(3, 1, 2, 2, 64, 128).cuda()
    pos = torch.tensor([bad, 63], dtype=torch.int32, device="cuda")
    out = Guarded((2, 4, 128), torch.bfloat16)
    T.window_decode_attn(Q, K, V, pos, 2, 16, 2, out=out.t)
    out.check("O")
    assert L.tp_get_device_status(check=False) == L.TP_ERR_SHAPE
    ref, tol = O.window_decode(f64(Q), f64(K), f64(V), [63, 63], 16, 2, SCALE)
    within(out.t[1], ref[1], tol[1])
    assert L.tp_get_device_status(check=False) == L.TP_OK


def test_two_graphs_share_a_workspace_one_after_the_other():
    heads, window, sink, L_max, B = (8, 2, 1), 40, 2, 200, 5
    K, V = rnd(2, 1, 2, B, L_max, 128).cuda(), rnd(3, 1, 2, B, L_max, 128).cuda()
    Qs = [rnd(s, B, 8, 128).cuda() for s in (5, 6)]
    pos = torch.tensor([199, 3, -1, 41, 42], dtype=torch.int32, device="cuda")
    ws = torch.empty(L.tp_window_decode_workspace_size(B, 8, 2, 128, 1), dtype=torch.uint8, device="cuda")
    outs = [torch.zeros(B, 8, 128, dtype=torch.bfloat16, device="cuda") for _ in Qs]
    want = [T.window_decode_attn(Q, K, V, pos, 2, window, sink, out=torch.zeros_like(outs[0])) for Q in Qs]
    torch.cuda.synchronize()
    graphs = []
    for Q, o in zip(Qs, outs):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            T.window_decode_attn(Q, K, V, pos, 2, window, sink, ws=ws, out=o)
        graphs.append(g)
    for _ in range(3):
        for g in graphs:
            g.replay()
    torch.cuda.synchronize()
    for o, w in zip(outs, want):
        assert torch.equal(o, w)


@pytest.mark.parametrize("rolling", [False, True])
def test_token_by_token_equals_the_packed_forward(rolling):
    """norm + rotation and window attention run over whole sequences, then token by token through the
    cache: the same numbers within both sides' bounds."""
    n_heads, n_kv, t = 8, 2, 2
    window, sink, lens = 21, 3, [60, 1, 37]
    N, B, Lc = sum(lens), len(lens), (24 if rolling else 60)
    X = rnd(1, t, N, O.tp_long_context.row_width(n_heads, n_kv, t), dtype=torch.bfloat16)
    gq, gk = [(1 + rnd(s, 128, std=0.2, dtype=torch.float32)).to(torch.bfloat16).cuda() for s in (2, 3)]
    f = T.rope_frequencies(128, 10000.0)
    pos = torch.tensor([p for n in lens for p in range(n)], dtype=torch.int32, device="cuda")
    cu = [0] + np.cumsum(lens).tolist()
    QKV = T.qk_norm_rope_forward(X.cuda(), n_heads, n_kv, gq, gk, 1e-6, f, pos)
    o, _ = T.window_attn_forward(QKV, n_heads, n_kv, window, sink, None,
                                 torch.tensor(cu, dtype=torch.int32, device="cuda"))
    # fp64 on the same rotated and rounded operands
    r = O.window_attention(f64(QKV), n_heads, n_kv, window, sink, SCALE, cu)
    within(o, r["O"], r["tol_O"])
    K, V = (torch.full((t, 1, B, Lc, 128), float("nan"), dtype=torch.float16, device="cuda") for _ in range(2))
    for step in range(max(lens)):
        p = torch.tensor([step if step < n else -1 for n in lens], dtype=torch.int32, device="cuda")
        rows = X[:, [cu[b] + min(step, lens[b] - 1) for b in range(B)]].contiguous().cuda()
        Q = T.qk_norm_rope_append(rows, n_heads, n_kv, K, V, p, gq, gk, 1e-6, f, window=window, n_sink=sink,
                                  rolling=rolling)
        got = T.window_decode_attn(Q, K, V, p, n_kv, window, sink, rolling=rolling)
        for b in range(B):
            if step < lens[b]:
                at = cu[b] + step
                # the append gives the forward's bits
                assert torch.equal(Q[b].view(t, 512), QKV[:, at, :512])
                within(got[b].view(t, 512), r["O"][:, at], r["tol_O"][:, at])
    assert L.tp_get_device_status(check=False) == L.TP_OK


def test_caches_past_32_bit_offsets():
    """Caches of 3e9 elements each: the last sequence's token is appended at its end and attends from there."""
    n_heads, n_kv, B, L_max, window, sink = 8, 1, 4, 6_000_000, 300, 4
    K, V = (torch.zeros(1, 1, B, L_max, 128, dtype=torch.float16, device="cuda") for _ in range(2))
    assert K.numel() > 2 ** 31
    pos = torch.tensor([-1, 5, L_max - 2, L_max - 1], dtype=torch.int32, device="cuda")
    seen = torch.cat([torch.arange(sink), torch.arange(L_max - window, L_max)]).cuda()
    Kc, Vc = rnd(2, 1, 1, 1, window + sink, 128), rnd(3, 1, 1, 1, window + sink, 128)
    K[:, :, 3, seen], V[:, :, 3, seen] = Kc[:, :, 0].cuda(), Vc[:, :, 0].cuda()
    X = rnd(1, 1, B, (n_heads + 2) * 128).cuda()
    Q = T.qk_norm_rope_append(X, n_heads, n_kv, K, V, pos, inv_freq=T.rope_frequencies(128))
    alone = T.qk_norm_rope_forward(X, n_heads, n_kv, inv_freq=T.rope_frequencies(128), pos=pos)[0, 3].view(-1, 128)
    assert torch.equal(Q[3], alone[:n_heads])
    assert torch.equal(K[0, 0, 3, -1], alone[n_heads]) and torch.equal(V[0, 0, 3, -1], alone[n_heads + 1])
    Kc[0, 0, 0, -1], Vc[0, 0, 0, -1] = alone[n_heads].cpu(), alone[n_heads + 1].cpu()
    ref, tol = O.window_decode(f64(Q[3:]), f64(Kc), f64(Vc), [window + sink - 1], window + sink, 0, SCALE, False)
    out = T.window_decode_attn(Q, K, V, pos, n_kv, window, sink, SCALE)
    within(out[3:], ref, tol)
    assert L.tp_get_device_status(check=False) == L.TP_OK


def test_positions_written_by_the_kernel_before():
    """A device kernel writes pos (another type's cast, an addition) directly before the call, eagerly and in a
    replayed graph: the result of positions that were there long before, bit for bit."""
    n_heads, n_kv, B, L_max, window, sink = 16, 2, 64, 2048, 300, 4
    Q, K, V = rnd(1, B, n_heads, 128).cuda(), rnd(2, 1, n_kv, B, L_max, 128).cuda(), rnd(3, 1, n_kv, B, L_max, 128).cuda()
    ws = torch.empty(L.tp_window_decode_workspace_size(B, n_heads, n_kv, 128, 1), dtype=torch.uint8, device="cuda")
    start = torch.randint(0, 900, (B,), generator=torch.Generator().manual_seed(4))
    start[7] = start[8] = -1
    steps = [start + 37 * k * (start >= 0) for k in range(1, 25)]
    want = []
    for p in steps:
        pos = p.to(torch.int32).cuda()
        torch.cuda.synchronize()
        want.append(T.window_decode_attn(Q, K, V, pos, n_kv, window, sink, out=torch.zeros_like(Q, dtype=torch.bfloat16)))
    torch.cuda.synchronize()
    add = (37 * (start >= 0)).to(torch.int32).cuda()
    out = torch.zeros(B, n_heads, 128, dtype=torch.bfloat16, device="cuda")
    pos = start.to(torch.int32).cuda()
    got = []
    for p in steps:
        pos.add_(add)
        got.append(T.window_decode_attn(Q, K, V, pos, n_kv, window, sink, ws=ws, out=out.clone()))
    assert all(torch.equal(g, w) for g, w in zip(got, want))
    long = torch.stack(steps).cuda()
    got = [T.window_decode_attn(Q, K, V, long[k].to(torch.int32), n_kv, window, sink, ws=ws, out=out.clone())
           for k in range(len(steps))]
    assert all(torch.equal(g, w) for g, w in zip(got, want))
    pos.copy_(start.to(torch.int32))
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pos.add_(add)
        T.window_decode_attn(Q, K, V, pos, n_kv, window, sink, ws=ws, out=out)
    got = []
    for _ in steps:
        graph.replay()
        got.append(out.clone())
    assert all(torch.equal(g, w) for g, w in zip(got, want))
    assert L.tp_get_device_status(check=False) == L.TP_OK


def test_a_batch_of_empty_rows_keeps_the_order_of_the_stream():
    """Kernels behind a decode step without work read what the kernels before it write: norm + rotation, an empty
    step, then the rotation in place on the result of the first, against the same calls with waits between."""
    n_heads, n_kv, N, B = 16, 2, 6000, 5
    X = rnd(1, 1, N, (n_heads + 2 * n_kv) * 128).cuda()
    f = T.rope_frequencies(128)
    Q, K, V = rnd(2, B, n_heads, 128).cuda(), rnd(3, 1, n_kv, B, 256, 128).cuda(), rnd(4, 1, n_kv, B, 256, 128).cuda()
    pos = torch.full((B,), -1, dtype=torch.int32, device="cuda")
    ws = torch.empty(L.tp_window_decode_workspace_size(B, n_heads, n_kv, 128, 1), dtype=torch.uint8, device="cuda")
    out, O_buf = torch.empty_like(X), torch.zeros(B, n_heads, 128, dtype=torch.bfloat16, device="cuda")

    def chain(wait):
        T.qk_norm_rope_forward(X, n_heads, n_kv, inv_freq=f, out=out)
        wait()
        T.window_decode_attn(Q, K, V, pos, n_kv, 100, 4, ws=ws, out=O_buf)
        wait()
        T.qk_norm_rope_forward(out, n_heads, n_kv, inv_freq=f, out=out)
        return out.clone()
    want = chain(torch.cuda.synchronize)
    for _ in range(20):
        out.zero_()
        assert torch.equal(chain(lambda: None), want)
    assert not O_buf.any()
    assert L.tp_get_device_status(check=False) == L.TP_OK
