"""Query / key norm with the rotary embedding on the GPU against the fp64 oracle: forward, backward and
the decode append, within bounds that count every rounding (oracle/tp_long_context.py)."""

import numpy as np
import pytest
import torch

import oracle as O
from gpu_helpers import Guarded, f64
from megatron_tensor_transformer_shard_gb300 import _lib as L
from megatron_tensor_transformer_shard_gb300 import tp as T

pytestmark = pytest.mark.gpu

HEADS = [(4, 2, 1), (8, 8, 2), (8, 2, 4), (64, 8, 8)]  # the third replicates KV heads


def width(n_heads, n_kv, t):
    return O.tp_long_context.row_width(n_heads, n_kv, t)


def rnd(seed, *shape, dtype=torch.float16, std=1.0):
    g = torch.Generator().manual_seed(seed)
    return (std * torch.randn(*shape, generator=g)).to(dtype)


def gammas(seed, norm):
    return [(1 + rnd(seed + k, 128, dtype=torch.float32, std=0.3)).to(torch.bfloat16) if norm else None
            for k in range(2)]


def cuda(*xs):
    return [None if x is None else x.cuda() for x in xs]


def np64(x):
    return None if x is None else f64(x)


def within(got, ref, tol):
    got = f64(got)
    assert got.shape == ref.shape
    bad = ~(np.abs(got - ref) <= tol)
    assert not bad.any(), (f"{bad.sum()} of {bad.size} off, first at {np.argwhere(bad)[0]}: "
                           f"{got[bad][0]} for {ref[bad][0]}, tolerance {tol[bad][0]}")


def positions(N, far):
    p = np.arange(N, dtype=np.int64) + far
    if N > 2:
        p[1], p[2] = 2 ** 31 - 1, -5
    return p


CASES = [  # heads, N, rot, norm, interleaved, bf16 input, first position
    (HEADS[0], 1, 128, True, False, False, 0), (HEADS[0], 3, 64, True, False, True, 100000),
    (HEADS[1], 37, 32, False, False, False, 0), (HEADS[2], 130, 128, True, True, True, 5000),
    (HEADS[2], 5, 16, False, True, False, 0), (HEADS[3], 67, 96, True, False, False, 70000),
    (HEADS[3], 9, 112, True, True, False, 0), (HEADS[0], 600, 0, True, False, False, 0),
]


@pytest.mark.parametrize("heads,N,rot,norm,inter,bf16,far", CASES)
def test_forward(heads, N, rot, norm, inter, bf16, far):
    n_heads, n_kv, t = heads
    X = rnd(1, t, N, width(*heads), dtype=torch.bfloat16 if bf16 else torch.float16, std=1.8)
    gq, gk = gammas(2, norm)
    f = T.rope_frequencies(rot, 500000.0, "cpu") if rot else None
    pos = torch.tensor(positions(N, far), dtype=torch.int32)
    ref, tol = O.qk_norm_rope(f64(X), n_heads, n_kv, np64(gq), np64(gk), 1e-5, None if f is None else f.numpy(),
                              pos.numpy(), inter)
    Xd, gqd, gkd, fd, pd = cuda(X, gq, gk, f, pos)
    out = Guarded(X.shape, torch.float16)
    T.qk_norm_rope_forward(Xd, n_heads, n_kv, gqd, gkd, 1e-5, fd, pd, inter, out=out.t)
    out.check("out")
    within(out.t, ref, tol)
    assert torch.equal(Xd.cpu().view(torch.int16), X.view(torch.int16))  # the input stays as it was
    again = T.qk_norm_rope_forward(Xd, n_heads, n_kv, gqd, gkd, 1e-5, fd, pd, inter)
    assert torch.equal(again.view(torch.int16), out.t.view(torch.int16))
    if not bf16:  # in place: the same bits, the values untouched
        T.qk_norm_rope_forward(Xd, n_heads, n_kv, gqd, gkd, 1e-5, fd, pd, inter, out=Xd)
        assert torch.equal(Xd.view(torch.int16), again.view(torch.int16))


def test_forward_default_positions_and_extreme_rows():
    n_heads, n_kv, t = 4, 2, 1
    N = 6
    X = rnd(1, t, N, width(4, 2, 1), dtype=torch.bfloat16)
    X[0, 1] = 0                                # an all-zero row: 0 with eps > 0
    X[0, 2] *= 2.0 ** 100                      # squares leave fp32
    X[0, 3] *= 2.0 ** -60                      # eps decides
    X[0, 4, 130] = float("nan")                # poisons its own head only
    X[0, 5, 5] = float("inf")
    gq, gk = gammas(2, True)
    f = T.rope_frequencies(128, device="cpu")
    Xv = X.clone()
    Xv[0, 2, 768:] = 1.0                       # the carried values stay within fp16
    X = Xv
    clean = f64(X)
    clean[0, 4, 130], clean[0, 5, 5] = 0, 0
    ref, tol = O.qk_norm_rope(clean, n_heads, n_kv, np64(gq), np64(gk), 1e-6, f.numpy())
    Y = f64(T.qk_norm_rope_forward(*cuda(X), n_heads, n_kv, *cuda(gq, gk), 1e-6, f.cuda()))
    heads = Y.reshape(N, -1, 128)
    assert np.isnan(heads[4, 1]).all() and np.isnan(heads[5, 0]).any()
    ok = np.ones(Y.shape, bool)
    ok[0, 4, 128:256] = ok[0, 5, :128] = False
    assert (np.abs(Y - ref)[ok] <= tol[ok]).all()


def units_bound(t, N, n_heads, n_kv):
    """Additions in the longest chain of a gamma gradient, in halves of fp32's last place: the heads that one
    of a warp's two groups visits (16 warps an SM, a unit of up to 6 heads more), 32 groups, the CTAs' sums by
    64, 6 levels; 56 for each term itself (24 as in the forward, the products, 16 of the phase)."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    per = n_heads // t + 2 * max(1, n_kv // t)
    visits = -(-t * N * per // (sms * 16 * 2)) + 6
    return (visits + 32 + sms / 64 + 6 + 56) * 2.0 ** -24


@pytest.mark.parametrize("f16_grad", [False, True])
@pytest.mark.parametrize("heads,N,rot,norm,inter,bf16,far", CASES)
def test_backward(heads, N, rot, norm, inter, bf16, far, f16_grad):
    n_heads, n_kv, t = heads
    X = rnd(1, t, N, width(*heads), dtype=torch.bfloat16 if bf16 else torch.float16, std=1.8)
    G = rnd(5, *X.shape, dtype=torch.float16 if f16_grad else torch.bfloat16)
    gq, gk = gammas(2, norm)
    f = T.rope_frequencies(rot, 500000.0, "cpu") if rot else None
    pos = torch.tensor(positions(N, far), dtype=torch.int32)
    dX, dq, dk, bX, bq, bk = O.qk_norm_rope_backward(f64(G), f64(X), n_heads, n_kv, np64(gq), np64(gk), 1e-5,
                                                     None if f is None else f.numpy(), pos.numpy(), inter)
    # 24 units as in the forward, twice (the norm's own factor), 12 of the dot product, 8 products; 16 of
    # the phase at position 2^31 (four fp64 roundings: 2^31 2^-51)
    half, sub = (2.0 ** -11, 2.0 ** -25) if f16_grad else (2.0 ** -8, 0.0)
    tol = half * np.abs(dX) + 84 * 2.0 ** -24 * bX + sub
    Xd, Gd, gqd, gkd, fd, pd = cuda(X, G, gq, gk, f, pos)
    out = Guarded(X.shape, G.dtype)
    args = (n_heads, n_kv, gqd, gkd, 1e-5, fd, pd, inter)
    got = T.qk_norm_rope_backward(Gd, Xd, *args, out=out.t)
    out.check("dX")
    within(out.t, dX, tol)
    if norm:
        units = units_bound(t, N, n_heads, n_kv)
        within(got[1], dq, units * bq)
        within(got[2], dk, units * bk)
        two = T.qk_norm_rope_backward(Gd, Xd, *args, grads=(got[1].clone(), got[2].clone()))
        within(two[1], 2 * dq, (2 * units + 2.0 ** -24) * bq + 2.0 ** -23 * np.abs(dq))
        again = T.qk_norm_rope_backward(Gd, Xd, *args)  # the same bits every time
        assert torch.equal(again[1], got[1]) and torch.equal(again[2], got[2])
    else:
        assert got[1] is None and got[2] is None
    T.qk_norm_rope_backward(Gd, Xd, *args, out=Gd)  # in place
    assert torch.equal(Gd.view(torch.int16), out.t.view(torch.int16))


def test_gamma_gradients_are_deterministic_over_many_rows():
    n_heads, n_kv, t, N = 64, 8, 4, 3001
    X = rnd(1, t, N, width(64, 8, 4)).cuda()
    G = rnd(2, *X.shape, dtype=torch.bfloat16).cuda()
    gq, gk = cuda(*gammas(3, True))
    f = T.rope_frequencies()
    a = T.qk_norm_rope_backward(G, X, n_heads, n_kv, gq, gk, inv_freq=f)
    b = T.qk_norm_rope_backward(G, X, n_heads, n_kv, gq, gk, inv_freq=f)
    assert torch.equal(a[1], b[1]) and torch.equal(a[2], b[2])
    _, dq, dk, _, bq, bk = O.qk_norm_rope_backward(f64(G), f64(X), n_heads, n_kv, f64(gq), f64(gk), 1e-6,
                                                   f.cpu().numpy())
    units = units_bound(t, N, n_heads, n_kv)
    within(a[1], dq, units * bq)
    within(a[2], dk, units * bk)


@pytest.mark.parametrize("rolling", [False, True])
@pytest.mark.parametrize("heads,B,rot,norm,bf16", [((4, 2, 1), 1, 128, True, True), ((8, 2, 4), 7, 64, False, False),
                                                   ((64, 8, 4), 33, 128, True, True), ((8, 8, 2), 5, 0, True, False)])
def test_append(heads, B, rot, norm, bf16, rolling):
    n_heads, n_kv, t = heads
    q_t, kv_t = O.tp_long_context.heads_of(n_heads, n_kv, t)
    window, sink, L_max = 11, 3, 17
    X = rnd(1, t, B, width(*heads), dtype=torch.bfloat16 if bf16 else torch.float16)
    gq, gk = gammas(2, norm)
    f = T.rope_frequencies(rot, 10000.0, "cpu") if rot else None
    top = 1000000 if rolling else L_max - 1
    pos = torch.tensor([top if b == 0 else (b * 7919) % (top + 1) for b in range(B)], dtype=torch.int32)
    if B > 3:
        pos[2] = -1
    ref, tol = O.qk_norm_rope(f64(X), n_heads, n_kv, np64(gq), np64(gk), 1e-6, None if f is None else f.numpy(),
                              pos.numpy())
    K, V = (Guarded((t, kv_t, B, L_max, 128), torch.float16) for _ in range(2))
    Q = Guarded((B, n_heads, 128), torch.float16)
    before = [c.t.clone() for c in (K, V, Q)]
    Xd, gqd, gkd, fd, pd = cuda(X, gq, gk, f, pos)
    T.qk_norm_rope_append(Xd, n_heads, n_kv, K.t, V.t, pd, gqd, gkd, 1e-6, fd, window=window, n_sink=sink,
                          rolling=rolling, out=Q.t)
    for name, c in (("K", K), ("V", V), ("Q", Q)):
        c.check(name)
    expect = [c.cpu() for c in before]
    for b in range(B):
        p = int(pos[b])
        if p < 0:
            assert torch.equal(Q.t[b].cpu().view(torch.int16), expect[2][b].view(torch.int16))
            continue
        slot = O.rolling_slot(p, window, sink) if rolling else p
        cols = slice(0, q_t * 128)
        within(Q.t[b].view(t, q_t * 128), ref[:, b, cols], tol[:, b, cols])
        for c, e, at in ((K, expect[0], q_t), (V, expect[1], q_t + kv_t)):
            cols = slice(at * 128, (at + kv_t) * 128)
            within(c.t[:, :, b, slot].reshape(t, -1), ref[:, b, cols], tol[:, b, cols])
            e[:, :, b, slot] = c.t[:, :, b, slot].cpu()
    for c, e in ((K, expect[0]), (V, expect[1])):  # every other slot as it was
        assert torch.equal(c.t.cpu().view(torch.int16), e.view(torch.int16))
    assert L.tp_get_device_status(check=False) == L.TP_OK


@pytest.mark.parametrize("bad", [-2, 17, 2 ** 31 - 1])
def test_append_reports_positions_past_the_cache(bad):
    X = rnd(1, 1, 2, width(4, 2, 1)).cuda()
    K, V = (torch.zeros(1, 2, 2, 17, 128, dtype=torch.float16, device="cuda") for _ in range(2))
    pos = torch.tensor([bad, 16], dtype=torch.int32, device="cuda")
    T.qk_norm_rope_append(X, 4, 2, K, V, pos, inv_freq=T.rope_frequencies())
    assert L.tp_get_device_status(check=False) == L.TP_ERR_SHAPE
    assert not K[:, :, 0].any() and not V[:, :, 0].any() and K[:, :, 1, 16].any()
    assert L.tp_get_device_status(check=False) == L.TP_OK


def test_two_streams_and_a_replayed_graph():
    n_heads, n_kv, t, N = 64, 8, 8, 50
    X = rnd(1, t, N, width(64, 8, 8)).cuda()
    gq, gk = cuda(*gammas(3, True))
    f = T.rope_frequencies()
    G = rnd(2, *X.shape, dtype=torch.bfloat16).cuda()
    want = T.qk_norm_rope_forward(X, n_heads, n_kv, gq, gk, inv_freq=f)
    wdx, wq, wk = T.qk_norm_rope_backward(G, X, n_heads, n_kv, gq, gk, inv_freq=f)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for st in streams:
        with torch.cuda.stream(st):
            got.append((T.qk_norm_rope_forward(X, n_heads, n_kv, gq, gk, inv_freq=f),
                        *T.qk_norm_rope_backward(G, X, n_heads, n_kv, gq, gk, inv_freq=f)))
    torch.cuda.synchronize()
    for y, dx, dq, dk in got:
        assert torch.equal(y, want) and torch.equal(dx, wdx) and torch.equal(dq, wq) and torch.equal(dk, wk)
    graph = torch.cuda.CUDAGraph()
    Xs, Gs = X.clone(), G.clone()
    with torch.cuda.graph(graph):
        y = T.qk_norm_rope_forward(Xs, n_heads, n_kv, gq, gk, inv_freq=f)
        dx, dq, dk = T.qk_norm_rope_backward(Gs, Xs, n_heads, n_kv, gq, gk, inv_freq=f)
    Xs.copy_(X.flip(1))
    Gs.copy_(G.flip(1))
    graph.replay()
    torch.cuda.synchronize()
    y2 = T.qk_norm_rope_forward(Xs, n_heads, n_kv, gq, gk, inv_freq=f)
    dx2, dq2, _ = T.qk_norm_rope_backward(Gs, Xs, n_heads, n_kv, gq, gk, inv_freq=f)
    assert torch.equal(y, y2) and torch.equal(dx, dx2) and torch.equal(dq, dq2)


def test_no_rows():
    z = torch.empty(2, 0, width(4, 2, 2), dtype=torch.float16, device="cuda")
    gq, gk = cuda(*gammas(1, True))
    assert T.qk_norm_rope_forward(z, 4, 2, gq, gk).shape == z.shape
    _, dq, dk = T.qk_norm_rope_backward(z, z.clone(), 4, 2, gq, gk)
    assert not dq.any() and not dk.any()
    one = torch.ones(128, device="cuda")
    T.qk_norm_rope_backward(z, z.clone(), 4, 2, gq, gk, grads=(one, one.clone()))
    assert (one == 1).all()


def test_rows_past_32_bit_offsets():
    """More than 2^31 elements: the last rows are what they are in a call of their own."""
    n_heads, n_kv, N, n = 64, 8, 220_000, 150
    R = width(n_heads, n_kv, 1)
    assert N * R > 2 ** 31
    gq, gk = cuda(*gammas(2, True))
    f = T.rope_frequencies(128)
    X, Y = (torch.zeros(1, N, R, dtype=torch.float16, device="cuda") for _ in range(2))
    X[:, N - n:], Y[:, N - n:] = rnd(1, 1, n, R).cuda(), rnd(3, 1, n, R).cuda()
    pos = torch.arange(N, dtype=torch.int32, device="cuda")
    kw = dict(q_gamma=gq, k_gamma=gk, inv_freq=f)
    out = T.qk_norm_rope_forward(X, n_heads, n_kv, pos=pos, **kw)
    tail = X[:, N - n:].clone(), Y[:, N - n:].clone(), pos[N - n:].clone()
    assert torch.equal(out[:, N - n:], T.qk_norm_rope_forward(tail[0], n_heads, n_kv, pos=tail[2], **kw))
    assert not out[:, :N - n].any()
    d, dq, dk = T.qk_norm_rope_backward(Y, X, n_heads, n_kv, pos=pos, **kw)
    d2, dq2, dk2 = T.qk_norm_rope_backward(tail[1], tail[0], n_heads, n_kv, pos=tail[2], **kw)
    assert torch.equal(d[:, N - n:], d2) and not d[:, :N - n].any()
    # The same terms g r x, and zeros, added in another order: each sum of m of them is off by at most m half steps of
    # the sum of their magnitudes, |g| <= |dy| + |dy of the pair's other half|.
    x, y = (v[0, :, :(n_heads + n_kv) * 128].view(n, -1, 128).double() for v in tail[:2])
    terms = (y.abs() + y.abs().roll(64, 2)) * x.abs() * (x.square().mean(2, keepdim=True) + 1e-6).rsqrt()
    for a, b, h in ((dq, dq2, slice(0, n_heads)), (dk, dk2, slice(n_heads, n_heads + n_kv))):
        m = n * (h.stop - h.start)
        assert ((a - b).abs() <= 2 * m * 2.0 ** -24 * terms[:, h].sum((0, 1))).all()
    assert L.tp_get_device_status(check=False) == L.TP_OK


def gamma_units(t, N, n_heads, n_kv):
    """Roundings in the longest chain of a gamma gradient, in halves of fp32's last place.  12 warps an SM share out
    the units, runs of up to 10 heads of a row (fewer when there are few rows); a 16-lane group adds up every second
    head of its units, then come 24 groups, every 64th CTA, 6 levels; and 56 for each term itself (24 as in the
    forward, the products, 16 of the phase)."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    per = n_heads // t + 2 * max(1, n_kv // t)
    chunks = max(-(-per // 10), min(per, -(-sms * 12 // (t * N))))
    heads = -(-per // chunks)
    chunks = -(-per // heads)
    visits = -(-t * N * chunks // (min(sms, t * N * chunks) * 12)) * -(-heads // 2)
    return (visits + 24 + -(-sms // 64) + 6 + 56) * 2.0 ** -24


def test_rows_of_any_magnitude_without_eps():
    """eps = 0: small rows, whose squares leave fp32 at the bottom, are normed like any other; zeros stay zeros, have
    no gradient and leave the gamma gradients alone."""
    n_heads, n_kv, t, N = 4, 2, 2, 12
    X = rnd(1, t, N, width(n_heads, n_kv, t), dtype=torch.bfloat16)
    G = rnd(5, *X.shape, dtype=torch.bfloat16)
    for row, e in ((1, -40), (2, -60), (3, -80), (4, -110), (5, -125), (6, 60)):
        X[:, row] *= 2.0 ** e
        G[:, row] *= 2.0 ** e                       # a gradient that leaves the result in bf16's range
    X[:, 7] = 0
    X[0, 8, 128:256] = 0                            # one head of a row
    X[:, :, 384:] = 1.0                             # the carried values
    gq, gk = gammas(2, True)
    f = T.rope_frequencies(128, 500000.0, "cpu")
    zero = np.zeros(X.shape, bool)
    zero[:, 7, :384] = zero[0, 8, 128:256] = True
    stand_in = f64(X)
    stand_in[zero] = 1.0                            # the oracle divides by 0 there
    ref, tol = O.qk_norm_rope(stand_in, n_heads, n_kv, f64(gq), f64(gk), 0.0, f.numpy())
    Xd, Gd, gqd, gkd, fd = cuda(X, G, gq, gk, f)
    Y = T.qk_norm_rope_forward(Xd, n_heads, n_kv, gqd, gkd, 0.0, fd)
    ref[zero] = 0
    within(Y, ref, tol)
    assert not Y.cpu().numpy()[zero].any()
    Gz = f64(G)
    Gz[zero] = 0                                    # no gradient through zeros
    dX, dq, dk, bX, bq, bk = O.qk_norm_rope_backward(Gz, stand_in, n_heads, n_kv, f64(gq), f64(gk), 0.0, f.numpy())
    # a rotated pair never mixes heads, so a zero head's gradient reaches nothing else
    got = T.qk_norm_rope_backward(Gd, Xd, n_heads, n_kv, gqd, gkd, 0.0, fd)
    dX[zero] = 0
    within(got[0], dX, 2.0 ** -8 * np.abs(dX) + 84 * 2.0 ** -24 * bX)
    units = gamma_units(t, N, n_heads, n_kv)
    within(got[1], dq, units * bq)
    within(got[2], dk, units * bk)
    K, V = (torch.zeros(t, 1, N, 16, 128, dtype=torch.float16, device="cuda") for _ in range(2))
    pos = torch.arange(N, dtype=torch.int32, device="cuda")
    Q = T.qk_norm_rope_append(Xd, n_heads, n_kv, K, V, pos, gqd, gkd, 0.0, fd)
    assert torch.equal(Q.view(N, t, 256).transpose(0, 1), Y[:, :, :256])
    assert torch.equal(K[:, 0, torch.arange(N), torch.arange(N)], Y[:, :, 256:384])


@pytest.mark.parametrize("n_heads,n_kv,t,N", [(64, 8, 4, 3001), (12, 4, 1, 20000), (8, 8, 2, 37)])
def test_gamma_gradients_within_the_longest_chain(n_heads, n_kv, t, N):
    X = rnd(1, t, N, width(n_heads, n_kv, t))
    G = rnd(2, *X.shape, dtype=torch.bfloat16)
    gq, gk = gammas(3, True)
    f = T.rope_frequencies(128, device="cpu")
    _, dq, dk, _, bq, bk = O.qk_norm_rope_backward(f64(G), f64(X), n_heads, n_kv, f64(gq), f64(gk), 1e-6, f.numpy())
    got = T.qk_norm_rope_backward(*cuda(G, X), n_heads, n_kv, *cuda(gq, gk), inv_freq=f.cuda())
    units = gamma_units(t, N, n_heads, n_kv)
    within(got[1], dq, units * bq)
    within(got[2], dk, units * bk)


@pytest.mark.parametrize("n_heads,n_kv,t,N", [(200, 1, 1, 3), (96, 96, 1, 70), (130, 65, 1, 1)])
def test_many_heads_a_shard(n_heads, n_kv, t, N):
    X = rnd(1, t, N, width(n_heads, n_kv, t))
    G = rnd(5, *X.shape, dtype=torch.bfloat16)
    gq, gk = gammas(2, True)
    f = T.rope_frequencies(64, device="cpu")
    ref, tol = O.qk_norm_rope(f64(X), n_heads, n_kv, f64(gq), f64(gk), 1e-6, f.numpy())
    args = (n_heads, n_kv, *cuda(gq, gk), 1e-6, f.cuda())
    within(T.qk_norm_rope_forward(X.cuda(), *args), ref, tol)
    dX, dq, dk, bX, bq, bk = O.qk_norm_rope_backward(f64(G), f64(X), n_heads, n_kv, f64(gq), f64(gk), 1e-6, f.numpy())
    got = T.qk_norm_rope_backward(G.cuda(), X.cuda(), *args)
    within(got[0], dX, 2.0 ** -8 * np.abs(dX) + 84 * 2.0 ** -24 * bX)
    units = gamma_units(t, N, n_heads, n_kv)
    within(got[1], dq, units * bq)
    within(got[2], dk, units * bk)
