"""Host-side checks of the long-context entry points: refused calls return their status before any device
work, and the Python layer names the wrong argument (no GPU needed)."""

import pytest
import torch

from megatron_tensor_transformer_shard_gb300 import _lib as L
from megatron_tensor_transformer_shard_gb300 import build as B
from megatron_tensor_transformer_shard_gb300 import tp as T

C = dict(check=False, stream=0)
P = 1 << 32  # a 16-byte aligned stand-in for a device pointer that no refused call reads


@pytest.fixture(scope="module", autouse=True)
def built_lib():
    B.build()
    return L.lib()


def fwd(x=P, N=4, nh=4, kv=2, hd=128, t=1, gq=P, gk=P, eps=1e-6, f=P, rot=128, pos=None, out=2 * P, flags=0):
    return L.tp_qk_norm_rope_forward(x, N, nh, kv, hd, t, gq, gk, eps, f, rot, pos, out, flags, **C)


def test_qk_norm_rope_forward_refusals():
    assert fwd(x=None) == fwd(out=None) == fwd(N=-1) == fwd(nh=0) == fwd(t=0) == L.TP_ERR_INVALID_ARG
    assert fwd(gq=None) == fwd(gk=None) == L.TP_ERR_INVALID_ARG               # one gamma without the other
    assert fwd(gq=None, gk=None, f=None) == L.TP_ERR_INVALID_ARG              # nothing to do
    assert fwd(eps=-1.0) == fwd(eps=float("nan")) == fwd(eps=float("inf")) == L.TP_ERR_INVALID_ARG
    assert fwd(hd=64) == fwd(nh=4, kv=3) == fwd(t=3) == fwd(nh=6, kv=3, t=2) == L.TP_ERR_SHAPE
    assert fwd(rot=0) == fwd(rot=8) == fwd(rot=24) == fwd(rot=144) == L.TP_ERR_SHAPE
    assert fwd(N=(1 << 30) + 1) == L.TP_ERR_SHAPE
    assert fwd(x=P + 8) == fwd(out=P + 8) == fwd(gq=P + 2) == fwd(f=P + 4) == fwd(pos=P + 2) == L.TP_ERR_ALIGN
    assert fwd(flags=8) == fwd(flags=L.TP_QKNR_F16_GRAD) == L.TP_ERR_UNSUPPORTED
    assert fwd(out=P + 16) == L.TP_ERR_INVALID_ARG                            # partly over its input
    assert fwd(x=None, out=None, N=0) == L.TP_OK


def test_qk_norm_rope_backward_refusals():
    ws = L.tp_qk_norm_rope_backward_workspace_size()

    def bwd(dy=P, x=2 * P, N=4, gq=P, gk=P, f=P, out=3 * P, dq=P, dk=P, flags=0, w=P, nws=ws):
        return L.tp_qk_norm_rope_backward(dy, x, N, 4, 2, 128, 1, gq, gk, 1e-6, f, 128, None, out, dq, dk, 0, flags,
                                          w, nws, **C)
    assert bwd(dy=None) == bwd(x=None) == bwd(out=None) == L.TP_ERR_INVALID_ARG
    assert bwd(gq=None, gk=None) == L.TP_ERR_INVALID_ARG                      # gamma gradients without a norm
    assert bwd(out=2 * P) == bwd(out=2 * P + 16) == bwd(out=P + 16) == L.TP_ERR_INVALID_ARG
    assert bwd(w=None) == bwd(nws=ws - 1) == L.TP_ERR_WORKSPACE
    assert bwd(w=P + 8) == bwd(dy=P + 8) == L.TP_ERR_ALIGN
    assert bwd(flags=16) == L.TP_ERR_UNSUPPORTED


def test_qk_norm_rope_append_refusals():
    def app(x=P, Bn=2, q=2 * P, k=4 * P, v=8 * P, Lm=64, pos=P, window=0, sink=0, rolling=0):
        return L.tp_qk_norm_rope_append(x, Bn, 4, 2, 128, 1, P, P, 1e-6, P, 128, pos, q, k, v, Lm, window, sink,
                                        rolling, 0, **C)
    assert app(x=None) == app(q=None) == app(k=None) == app(v=None) == app(pos=None) == L.TP_ERR_INVALID_ARG
    assert app(Lm=0) == app(window=0, rolling=1) == app(window=4, sink=-1, rolling=1) == L.TP_ERR_INVALID_ARG
    big = (1 << 63) - 1
    assert app(window=61, sink=4, rolling=1) == app(window=big, sink=1, rolling=1) == L.TP_ERR_SHAPE
    assert app(window=1, sink=big, rolling=1) == app(Lm=(1 << 30) + 1) == L.TP_ERR_SHAPE
    assert app(k=4 * P + 8) == app(q=2 * P + 8) == L.TP_ERR_ALIGN
    assert app(v=4 * P) == app(q=4 * P) == app(x=2 * P) == app(x=8 * P) == app(v=4 * P + 1024) == L.TP_ERR_INVALID_ARG  # overlaps
    assert app(x=None, Bn=0) == L.TP_OK


def test_python_layer_names_the_wrong_argument():
    x = torch.zeros(2, 3, 512, dtype=torch.float16)
    f = T.rope_frequencies(128, device="cpu")
    g = torch.ones(128, dtype=torch.bfloat16)
    for kw, what in [(dict(inv_freq=f.float()), "inv_freq"), (dict(q_gamma=g), "go together"), (dict(), "neither"),
                     (dict(inv_freq=f[:5]), "rotary"), (dict(inv_freq=f, pos=torch.zeros(4, dtype=torch.int32)), "pos"),
                     (dict(inv_freq=f, pos=torch.zeros(3)), "pos")]:
        with pytest.raises(ValueError, match=what):
            T.qk_norm_rope_forward(x, 4, 2, **kw)
    with pytest.raises(ValueError, match="row width"):
        T.qk_norm_rope_forward(x, 8, 2, inv_freq=f)
    with pytest.raises(ValueError, match="contiguous"):
        T.qk_norm_rope_forward(torch.zeros(2, 6, 512, dtype=torch.float16)[:, ::2], 4, 2, inv_freq=f)
    with pytest.raises(ValueError, match="dtype"):
        T.qk_norm_rope_forward(x.float(), 4, 2, inv_freq=f)
    with pytest.raises(ValueError, match="do not split"):
        T.qk_norm_rope_forward(x, 6, 4, inv_freq=f)


def wfwd(x=P, N=4, d=512, nh=4, kv=2, hd=128, t=1, W=8, S=0, cu=None, n=0, o=2 * P, lse=4 * P, ws=None, nws=0):
    return L.tp_attn_window_forward(x, N, d, nh, kv, hd, t, W, S, 0.1, cu, n, o, lse, ws, nws, **C)


def test_window_forward_refusals():
    assert wfwd(x=None) == wfwd(o=None) == wfwd(lse=None) == wfwd(N=-1) == wfwd(t=0) == L.TP_ERR_INVALID_ARG
    assert wfwd(W=0) == wfwd(W=-1) == wfwd(S=-1) == L.TP_ERR_INVALID_ARG
    assert wfwd(cu=P) == wfwd(n=2) == wfwd(cu=P, n=-1) == L.TP_ERR_INVALID_ARG       # boundaries and count go together
    assert wfwd(hd=64) == wfwd(d=500) == wfwd(kv=3) == wfwd(t=3) == L.TP_ERR_SHAPE
    assert wfwd(N=(1 << 30) + 1) == wfwd(cu=P, n=(1 << 30) + 1) == L.TP_ERR_SHAPE
    assert wfwd(x=P + 8) == wfwd(o=P + 8) == wfwd(cu=P + 2, n=2) == L.TP_ERR_ALIGN
    need = L.tp_attn_window_forward_workspace_size(4, 2)
    assert need >= 256 + 4 * 8 and L.tp_attn_window_forward_workspace_size(4, 0) == 0
    assert wfwd(cu=P, n=2) == wfwd(cu=P, n=2, ws=P, nws=need - 1) == L.TP_ERR_WORKSPACE
    assert wfwd(cu=P, n=2, ws=P + 16, nws=need) == L.TP_ERR_ALIGN
    # over the input, or each other
    assert wfwd(o=P + 64) == wfwd(o=P) == wfwd(lse=P + 4) == wfwd(lse=2 * P + 4) == L.TP_ERR_INVALID_ARG
    assert wfwd(N=(1 << 29) + 1) == L.TP_ERR_SHAPE
    assert wfwd(x=None, o=None, lse=None, N=0) == L.TP_OK


def test_window_backward_refusals():
    size = L.tp_attn_window_backward_workspace_size

    def bwd(x=P, dx=2 * P, D=16 * P, N=4, W=8, S=0, cu=None, n=0, flags=0, ws=None, nws=0):
        return L.tp_attn_window_backward(x, 4 * P, 8 * P, 32 * P, N, 512, 4, 2, 128, 1, W, S, 0.1, cu, n, D, dx, flags,
                                         ws, nws, **C)
    assert bwd(x=None) == bwd(dx=None) == bwd(D=None) == bwd(W=0) == L.TP_ERR_INVALID_ARG
    assert bwd(dx=P + 8) == L.TP_ERR_ALIGN and bwd(flags=2) == L.TP_ERR_UNSUPPORTED
    assert bwd(dx=P) == bwd(dx=4 * P) == bwd(dx=8 * P + 16) == bwd(dx=32 * P) == L.TP_ERR_INVALID_ARG  # over an input
    assert bwd(D=P) == bwd(D=4 * P) == bwd(D=8 * P) == bwd(D=32 * P + 4) == bwd(D=2 * P) == L.TP_ERR_INVALID_ARG
    assert size(4, 512, 4, 2, 128, 1, 8, 2, 0) == 0                       # no query beyond a window's reach
    need = size(1000, 512, 4, 2, 128, 1, 8, 2, 0)
    assert need == 2 * 16 * 2 * 2 * 128 * 4         # KV heads, chunks of 128 rows twice, sinks, dV and dK
    assert size(1000, 512, 4, 2, 128, 1, 8, 2, 3) == need + 256 + 8192    # and the rows' sequences
    assert size(1000, 512, 4, 2, 64, 1, 8, 2, 0) == size(-1, 512, 4, 2, 128, 1, 8, 2, 0) == 0
    assert bwd(N=1000, S=2) == bwd(N=1000, S=2, ws=P, nws=need - 1) == L.TP_ERR_WORKSPACE
    assert bwd(N=1000, S=2, ws=P + 16, nws=need) == L.TP_ERR_ALIGN


def test_window_python_layer_names_the_wrong_argument():
    x = torch.zeros(1, 8, 512, dtype=torch.float16)
    for kw, what in [(dict(window=0), "window"), (dict(window=4, n_sink=-1), "n_sink"),
                     (dict(cu_seqlens=torch.zeros(3)), "cu_seqlens"),
                     (dict(cu_seqlens=torch.zeros(1, dtype=torch.int32)), "cu_seqlens"),
                     (dict(out=torch.zeros(1, 8, 256)), "out"), (dict(lse=torch.zeros(1, 2, 7)), "lse")]:
        with pytest.raises(ValueError, match=what):
            T.window_attn_forward(x, 2, 1, **kw)
    with pytest.raises(ValueError, match="dtype"):
        T.window_attn_forward(x.bfloat16(), 2, 1)


def test_window_decode_refusals():
    need = L.tp_window_decode_workspace_size(2, 4, 2, 128, 1)
    assert need > 0 and L.tp_window_decode_workspace_size(2, 4, 2, 64, 1) == 0

    def dec(q=P, Bn=2, nh=4, kv=2, hd=128, t=1, W=8, S=0, roll=0, k=P, v=P, Lm=64, pos=P, o=P, ws=P, nws=need):
        return L.tp_window_decode_forward(q, Bn, nh, kv, hd, t, W, S, roll, 0.1, k, v, Lm, pos, o, ws, nws, **C)
    assert dec(q=None) == dec(k=None) == dec(v=None) == dec(pos=None) == dec(o=None) == L.TP_ERR_INVALID_ARG
    assert dec(W=0) == dec(S=-1) == dec(Lm=0) == dec(Bn=-1) == L.TP_ERR_INVALID_ARG
    assert dec(hd=64) == dec(kv=3) == dec(t=3) == dec(Bn=257) == dec(nh=64, kv=1) == L.TP_ERR_SHAPE
    assert dec(W=60, S=5, roll=1) == dec(W=(1 << 63) - 1, S=1, roll=1) == dec(Lm=(1 << 30) + 1) == L.TP_ERR_SHAPE
    assert dec(Bn=256, Lm=1 << 25) == L.TP_ERR_SHAPE                       # more tiles than the list can index
    assert dec(q=P + 8) == dec(o=P + 8) == dec(k=P + 8) == dec(pos=P + 1) == dec(ws=P + 16) == L.TP_ERR_ALIGN
    assert dec(ws=None) == dec(nws=need - 1) == L.TP_ERR_WORKSPACE
    assert dec(q=None, Bn=0) == L.TP_OK


def test_window_decode_python_layer_names_the_wrong_argument():
    q = torch.zeros(2, 4, 128, dtype=torch.float16)
    kv = torch.zeros(1, 2, 2, 16, 128, dtype=torch.float16)
    pos = torch.zeros(2, dtype=torch.int32)
    for args, kw, what in [((q, kv, kv, pos.long(), 2), {}, "pos"), ((q, kv, kv[:, :, :1], pos, 2), {}, "V_cache"),
                           ((q, kv, kv, pos, 4), {}, "row width"), ((q, kv, kv, pos, 2), dict(rolling=True), "rolling"),
                           ((q.bfloat16(), kv, kv, pos, 2), {}, "dtype"), ((q, kv, kv, pos, 2), dict(window=0), "window")]:
        with pytest.raises(ValueError, match=what):
            T.window_decode_attn(*args, **kw)


def opts(**kw):
    o = L.AttnOptions()
    for k, v in kw.items():
        setattr(o, k, v)
    opts.keep = o  # alive until the next one
    import ctypes
    return ctypes.addressof(o)


def test_attention_option_refusals():
    def fwd_(o, x=P, N=4, d=512, raw=None, q=2 * P, ws=None, nws=0, flags=0):
        return L.tp_attn_opt_forward(x, N, d, 4, 2, 128, 1, 0.1, o, P, None, P, None, None, P, raw, q, P, P, flags, ws,
                                     nws, **C)
    ok = dict(window=8, n_sink=2, inv_freq=P, rot_dim=64)
    assert fwd_(None) == fwd_(opts(window=-1)) == fwd_(opts(n_sink=-1)) == L.TP_ERR_INVALID_ARG
    assert fwd_(opts(q_gamma=P)) == fwd_(opts(cu_seqlens=P)) == fwd_(opts(n_seq=1)) == L.TP_ERR_INVALID_ARG
    assert fwd_(opts(**ok), raw=2 * P) == fwd_(opts(window=8), raw=P) == L.TP_ERR_INVALID_ARG
    assert fwd_(opts(inv_freq=P, rot_dim=40)) == fwd_(opts(**ok), d=500) == L.TP_ERR_SHAPE
    assert fwd_(opts(flags=1)) == fwd_(opts(**ok), flags=2) == L.TP_ERR_UNSUPPORTED
    assert fwd_(opts(**ok), q=P + 8) == fwd_(opts(**ok), ws=P + 16, nws=64) == L.TP_ERR_ALIGN
    assert fwd_(opts(cu_seqlens=P, n_seq=2)) == L.TP_ERR_WORKSPACE
    assert fwd_(opts(**ok), x=None) == L.TP_ERR_INVALID_ARG and fwd_(opts(**ok), N=0) == L.TP_OK
    size = L.tp_attn_opt_backward_workspace_size
    norm = dict(ok, q_gamma=P, k_gamma=P, eps=1e-6)
    need = size(300, 512, 4, 2, 128, 1, opts(**norm))
    assert need > size(300, 512, 4, 2, 128, 1, opts(**ok)) > size(300, 512, 4, 2, 128, 1, opts()) > 0
    assert size(300, 512, 4, 2, 128, 1, opts(window=-1)) == 0

    def bwd(o, raw=P, dqg=None, ws=P, nws=need):
        return L.tp_attn_opt_backward(P, P, raw, P, P, P, 300, 512, 4, 2, 128, 1, 0.1, o, P, P, P, P, P, P, P, dqg, None,
                                      0, 0, ws, nws, **C)
    assert bwd(opts(**norm), raw=None) == bwd(opts(**ok), dqg=P) == L.TP_ERR_INVALID_ARG
    assert bwd(opts(**norm), ws=None) == bwd(opts(**norm), nws=4096) == L.TP_ERR_WORKSPACE
    assert bwd(opts(**norm), ws=P + 16) == L.TP_ERR_ALIGN


def test_decode_attention_option_refusals():
    need = L.tp_decode_attn_opt_workspace_size(2, 512, 4, 2, 128, 1)
    assert need > 0 and L.tp_decode_attn_opt_workspace_size(2, 512, 4, 2, 64, 1) == 0

    def dec(o, x=P, Bn=2, Lm=64, ws=P, nws=need):
        return L.tp_decode_attn_opt_forward(x, Bn, 512, 4, 2, 128, 1, 0.1, o, P, None, P, None, P, P, Lm, P, P, ws, nws, **C)
    ok = dict(window=8, n_sink=2, inv_freq=P, rot_dim=64)
    assert dec(None) == dec(opts(rolling=1)) == dec(opts(k_gamma=P)) == dec(opts(**ok), x=None) == L.TP_ERR_INVALID_ARG
    assert dec(opts(window=64, n_sink=1, rolling=1)) == dec(opts(inv_freq=P, rot_dim=8)) == L.TP_ERR_SHAPE
    assert dec(opts(**ok), nws=need - 1) == L.TP_ERR_WORKSPACE and dec(opts(**ok), ws=P + 16) == L.TP_ERR_ALIGN
    assert dec(opts(flags=2)) == L.TP_ERR_UNSUPPORTED and dec(opts(**ok), x=None, Bn=0) == L.TP_OK


def test_attention_options_name_the_wrong_argument():
    g = torch.ones(128, dtype=torch.bfloat16)
    f = T.rope_frequencies(128, device="cpu")
    for kw, what in [(dict(window=0), "window"), (dict(n_sink=-1), "n_sink"), (dict(q_gamma=g), "go together"),
                     (dict(rolling=True), "rolling"), (dict(inv_freq=f[:4]), "rotary"), (dict(inv_freq=f.float()), "inv_freq"),
                     (dict(cu_seqlens=torch.zeros(1, dtype=torch.int32)), "cu_seqlens"),
                     (dict(pos=torch.zeros(2, 2, dtype=torch.int32)), "pos")]:
        with pytest.raises(ValueError, match=what):
            T.AttentionOptions(**kw)


def test_sinks_that_hide_nothing_take_no_workspace():
    """window + n_sink >= N is full causal attention: no partial sums of sinks, however many there are."""
    def size(N, W, S, n_seq=0):
        return L.tp_attn_window_backward_workspace_size(N, 64 * 128, 64, 8, 128, 1, W, S, n_seq)
    for S in (16384, 10 ** 9, 2 ** 62, 16384 - 1):
        assert size(16384, 1, S) == 0
    assert size(16384, 1024, 16384 - 1024) == 0 and size(16384, 1024, 16384) == 0
    assert size(16384, 1024, 16384, 3) == 256 + 8 * 16384      # the rows' sequences alone
    assert size(16384, 1, 16382) > 0 and size(16384, 1024, 16384 - 1025) > 0
    assert size(1, 1, 1) == size(0, 1, 10 ** 9) == 0


def test_blocks_check_the_buffers_of_out():
    """A short, wrongly typed or missing buffer is named before anything is launched."""
    import types
    bf, N, d = torch.bfloat16, 6, 512
    X, W, Wo = torch.zeros(N, d, dtype=bf), torch.zeros(1, 1024, d, dtype=bf), torch.zeros(1, d, 512, dtype=bf)
    opt = T.AttentionOptions(4)
    good = dict(Y=torch.zeros(N, d, dtype=bf), QKV=torch.zeros(1, N, 1024, dtype=torch.float16),
                O=torch.zeros(1, N, 512, dtype=bf), lse=torch.zeros(1, 4, N))

    def fwd_(**kw):
        with pytest.raises(ValueError) as e:
            T.attn_opt_forward(X, W, None, Wo, None, 4, 2, 1, opt, out=tuple({**good, **kw}.values()))
        return str(e.value)
    for kw in (dict(Y=good["Y"][:5]), dict(Y=good["Y"].half()), dict(Y=None), dict(QKV=good["QKV"].bfloat16()),
               dict(QKV=good["QKV"][:, :, :512]), dict(O=torch.zeros(1, N, 256, dtype=bf)), dict(lse=good["lse"].half()),
               dict(lse=torch.zeros(4, N))):
        assert f"{next(iter(kw))} of out" in fwd_(**kw)
    assert "buffers" in fwd_(more=good["Y"])
    grads = dict(dX=good["Y"], dWqkv=torch.zeros(1, 1024, d), dbqkv=torch.zeros(1, 1024), dWo=torch.zeros(1, d, 512),
                 dbo=torch.zeros(d))

    def bwd(attn=opt, raw=None, **kw):
        with pytest.raises(ValueError) as e:
            T.attn_opt_backward(X, X, raw, good["QKV"], good["O"], good["lse"], W, Wo, 4, 2, 1, attn,
                                out=tuple({**grads, **kw}.values()))
        return str(e.value)
    for kw in (dict(dX=X.float()), dict(dWqkv=grads["dWqkv"][:, :512]), dict(dWqkv=W), dict(dbqkv=torch.zeros(512)),
               dict(dWo=torch.zeros(d, 512)), dict(dbo=torch.zeros(4)), dict(dX=None)):
        assert f"{next(iter(kw))} of out" in bwd(**kw)
    g = torch.ones(128, dtype=bf)
    assert "QKV_raw" in bwd(T.AttentionOptions(4, q_gamma=g, k_gamma=g))
    w = types.SimpleNamespace(t=1, kv_t=2, d=d, n_heads=4, n_kv=2, head_dim=128)
    cache = torch.zeros(1, 2, 3, 8, 128, dtype=torch.float16)
    for out in (torch.zeros(2, d, dtype=bf), torch.zeros(3, d), torch.zeros(3, 2 * d, dtype=bf)[:, ::2]):
        with pytest.raises(ValueError, match="out"):
            T.decode_attn_forward(X[:3], w, cache, cache.clone(), torch.zeros(3, dtype=torch.int32), attn=opt, out=out)
    ws = torch.zeros(64, dtype=torch.uint8, device="meta")
    with pytest.raises(ValueError, match="ws is on"):
        T.decode_attn_forward(X[:3], w, cache, cache.clone(), torch.zeros(3, dtype=torch.int32), attn=opt, ws=ws)
    with pytest.raises(ValueError, match="ws is on"):
        T.window_decode_attn(torch.zeros(3, 4, 128, dtype=torch.float16), cache, cache.clone(),
                             torch.zeros(3, dtype=torch.int32), 2, 4, ws=ws)


def test_blocks_refuse_before_they_launch():
    """What a block's later steps refuse is refused before its first: here a launch would give TP_ERR_CUDA."""
    ok = dict(window=8, n_sink=2, inv_freq=P, rot_dim=64)
    need = L.tp_decode_attn_opt_workspace_size(2, 512, 4, 2, 128, 1)

    def dec(x=P, k=2 * P, v=4 * P, pos=8 * P, y=16 * P, ws=32 * P, o=None):
        return L.tp_decode_attn_opt_forward(x, 2, 512, 4, 2, 128, 1, 0.1, o or opts(**ok), P, None, P, None, k, v, 64, pos, y,
                                            ws, need, **C)
    cache = 2 * 2 * 64 * 128 * 2
    assert dec(k=4 * P) == dec(v=2 * P + cache - 256) == L.TP_ERR_INVALID_ARG          # the caches over each other
    assert dec(k=32 * P) == dec(v=32 * P - cache + 256) == L.TP_ERR_INVALID_ARG        # over the workspace
    assert dec(pos=8 * P + 2) == L.TP_ERR_ALIGN

    def fwd_(raw=None, q=2 * P, O=4 * P, lse=8 * P, N=40, ws=None, nws=0, **o):
        return L.tp_attn_opt_forward(P, N, 512, 4, 2, 128, 1, 0.1, opts(**{**ok, **o}), P, None, P, None, None, 16 * P, raw, q,
                                     O, lse, 0, ws, nws, **C)
    assert fwd_(raw=2 * P + 16) == fwd_(raw=2 * P - 1024) == L.TP_ERR_INVALID_ARG       # the raw rows partly over the rotated
    assert fwd_(O=2 * P + 1024) == fwd_(lse=2 * P + 64) == fwd_(lse=4 * P + 64) == L.TP_ERR_INVALID_ARG
    assert fwd_(N=(1 << 29) + 1) == L.TP_ERR_SHAPE

    def bwd(raw=64 * P, qkv=2 * P, O=4 * P, lse=8 * P, ws=32 * P, N=40):
        o = opts(**ok, q_gamma=P, k_gamma=P, eps=1e-6)
        return L.tp_attn_opt_backward(16 * P, P, raw, qkv, O, lse, N, 512, 4, 2, 128, 1, 0.1, o, P, P, 128 * P, 256 * P, None,
                                      256 * P, None, None, None, 0, 0, ws, 1 << 62, **C)
    inside = 32 * P + 4096
    assert bwd(qkv=inside) == bwd(O=inside) == bwd(lse=inside) == bwd(raw=inside) == L.TP_ERR_INVALID_ARG
    assert bwd(N=(1 << 29) + 1) == L.TP_ERR_SHAPE


def test_window_decode_refuses_overlaps():
    need = L.tp_window_decode_workspace_size(2, 4, 2, 128, 1)
    qb, cache = 2 * 4 * 128 * 2, 2 * 2 * 64 * 128 * 2

    def dec(q=P, k=2 * P, v=4 * P, pos=8 * P, o=16 * P, ws=32 * P):
        return L.tp_window_decode_forward(q, 2, 4, 2, 128, 1, 8, 0, 0, 0.1, k, v, 64, pos, o, ws, need, **C)
    assert dec(o=P) == dec(o=P + qb - 16) == dec(o=P - qb + 16) == L.TP_ERR_INVALID_ARG                # the queries
    assert dec(o=2 * P + cache - 16) == dec(o=4 * P) == dec(o=8 * P) == L.TP_ERR_INVALID_ARG           # caches, positions
    assert dec(o=32 * P + 256) == dec(o=32 * P - 256) == L.TP_ERR_INVALID_ARG                          # the workspace
    assert dec(q=32 * P + 256) == dec(k=32 * P) == dec(v=32 * P - 256) == dec(pos=32 * P + need - 4) == L.TP_ERR_INVALID_ARG
    ok = dict(window=8, n_sink=2)
    total = L.tp_decode_attn_opt_workspace_size(2, 512, 4, 2, 128, 1)

    def step(x=P, k=2 * P, v=4 * P, y=16 * P, ws=32 * P):
        return L.tp_decode_attn_opt_forward(x, 2, 512, 4, 2, 128, 1, 0.1, opts(**ok), P, None, P, None, k, v, 64, 8 * P, y, ws,
                                            total, **C)
    assert step(y=2 * P) == step(y=4 * P + cache - 16) == step(y=32 * P + total - 16) == L.TP_ERR_INVALID_ARG
    assert step(x=32 * P + total - 16) == step(k=32 * P + total - 256) == L.TP_ERR_INVALID_ARG


def test_fp32_pointers_between_words_are_refused():
    assert wfwd(lse=4 * P + 2) == L.TP_ERR_ALIGN

    def wbwd(lse=32 * P, D=16 * P):
        return L.tp_attn_window_backward(P, 4 * P, 8 * P, lse, 4, 512, 4, 2, 128, 1, 8, 0, 0.1, None, 0, D, 2 * P, 0, None, 0,
                                         **C)
    assert wbwd(lse=32 * P + 2) == wbwd(D=16 * P + 1) == L.TP_ERR_ALIGN

    def nbwd(N=4, dq=P, dk=P):
        return L.tp_qk_norm_rope_backward(P, 2 * P, N, 4, 2, 128, 1, P, P, 1e-6, P, 128, None, 4 * P, dq, dk, 0, 0, P,
                                          L.tp_qk_norm_rope_backward_workspace_size(), **C)
    assert nbwd(dq=P + 2) == nbwd(dk=P + 1) == nbwd(N=0, dq=P + 2) == L.TP_ERR_ALIGN
