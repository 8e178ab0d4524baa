"""CPU pins of the windowed-attention reference (oracle/sink.py), and the
refusals of the entry points that compute it."""
import ctypes

import numpy as np
import pytest
import torch

import oracle
from long_context_causal_gb300 import dfa
from oracle import sink

lib = dfa.library()
A = 0x10000          # an aligned stand-in address: validation fails before any use
MIS = 0x10008        # not 16-byte aligned


def draw(B, S, H, Hkv, D, seed=0):
    r = np.random.default_rng(seed)
    return (r.standard_normal((B, S, H, D)), r.standard_normal((B, S, Hkv, D)), r.standard_normal((B, S, Hkv, D)),
            r.standard_normal((B, S, H, D)))


def test_a_window_over_every_key_is_causal_attention():
    q, k, v, do = draw(2, 37, 4, 2, 16)
    O, lse, size = sink.attn_fwd(q, k, v, 37, 0)
    Or, lr = oracle.attn_fwd(q, k, v)
    assert np.allclose(O, Or, atol=1e-13) and np.allclose(lse, lr, atol=1e-13) and (size >= np.abs(O) - 1e-15).all()
    got = sink.attn_bwd(q, k, v, O, lse, do, 1000, 5)
    for name, ref in zip(("dQ", "dK", "dV"), oracle.attn_bwd(q, k, v, do)):
        assert np.allclose(got[name][0], ref, atol=1e-12), name
        assert (got[name][1] >= np.abs(ref) - 1e-13).all(), name


@pytest.mark.parametrize("window,n_sink", [(1, 0), (1, 3), (5, 0), (5, 2), (20, 7), (40, 40)])
def test_masked_library_attention_and_its_autograd_agree(window, n_sink):
    S, D = 40, 8
    q, k, v, do = draw(1, S, 2, 1, D, seed=3)
    i, j = torch.arange(S)[:, None], torch.arange(S)
    mask = (j <= i) & ((j > i - window) | (j < n_sink))
    tq, tk, tv = (torch.tensor(t).transpose(1, 2).requires_grad_() for t in (q, k, v))
    out = torch.nn.functional.scaled_dot_product_attention(tq, tk.expand(1, 2, S, D), tv.expand(1, 2, S, D),
                                                           attn_mask=mask)
    out.backward(torch.tensor(do).transpose(1, 2))
    O, lse, _ = sink.attn_fwd(q, k, v, window, n_sink)
    assert np.allclose(O, out.detach().transpose(1, 2).numpy(), atol=1e-13)
    got = sink.attn_bwd(q, k, v, O, lse, do, window, n_sink)
    for name, t in (("dQ", tq), ("dK", tk), ("dV", tv)):
        assert np.allclose(got[name][0], t.grad.transpose(1, 2).numpy(), atol=1e-12), name


def test_gradients_are_the_forwards_differences():
    q, k, v, do = draw(1, 9, 2, 1, 4, seed=5)
    O, lse, _ = sink.attn_fwd(q, k, v, 3, 2)
    got = sink.attn_bwd(q, k, v, O, lse, do, 3, 2)
    f = lambda *t: float((sink.attn_fwd(*t, 3, 2)[0] * do).sum())  # noqa: E731
    for z, name in enumerate(("dQ", "dK", "dV")):
        args = [q.copy(), k.copy(), v.copy()]
        num = np.zeros_like(args[z])
        for at in np.ndindex(num.shape):
            x = args[z][at]
            args[z][at] = x + 1e-6
            up = f(*args)
            args[z][at] = x - 1e-6
            num[at] = (up - f(*args)) / 2e-6
            args[z][at] = x
        assert np.allclose(got[name][0], num, atol=1e-8), name


def test_decode_is_the_forwards_last_row():
    q, k, v, _ = draw(2, 33, 4, 2, 8, seed=7)
    for n in (1, 6, 33):
        O, lse, _ = sink.attn_fwd(q[:, :n], k[:, :n], v[:, :n], 5, 3)
        Od, ld, _ = sink.decode(q[:, n - 1], k, v, [n, n], 5, 3)
        assert np.allclose(Od, O[:, -1], atol=1e-13) and np.allclose(ld, lse[:, :, -1], atol=1e-13)
    O, lse, _ = sink.decode(q[:, 0], k, v, [0, 0], 5, 3)
    assert (O == 0).all() and (lse == -np.inf).all()


def test_checkpoint_values():
    x = np.zeros((1, 64))
    x[0, :4] = [1.0, -0.5, 1 / 128, 0.25]        # exponent 0: steps of 2^-6; 1/128 is half a step and goes to 0
    x[0, 32:34] = [1.9921875, 127.5 / 64 / 2]    # 255/128: 127.5 steps, held as 127
    y = sink.ckpt8(x)
    assert (y[0, :4] == [1.0, -0.5, 0.0, 0.25]).all() and y[0, 32] == 127 / 64 and y[0, 33] == 64 / 64
    r = np.random.default_rng(1).standard_normal((7, 3, 128)) * 10.0 ** np.arange(-3, 4)[:, None, None]
    bf = torch.tensor(r).bfloat16().double().numpy()
    y = sink.ckpt8(bf)
    big = np.abs(bf.reshape(7, 3, 4, 32)).max(-1, keepdims=True)
    step = 2.0 ** (np.floor(np.log2(big)) - 6)
    # half a step, and at most one at 127.5 steps or above
    assert (np.abs(y - bf).reshape(7, 3, 4, 32) <= np.where(np.abs(bf.reshape(7, 3, 4, 32)) > 127 * step, 1, 0.5) * step).all()
    assert (torch.tensor(y).bfloat16().double().numpy() == y).all()      # bf16 numbers
    assert (sink.ckpt8(y) == y).all()                                    # held again, they stay
    bad = r[0].copy()
    bad[1, 40] = np.inf
    bad[2, 5] = np.nan
    y = sink.ckpt8(bad)
    assert np.isnan(y[1, 32:64]).all() and np.isnan(y[2, :32]).all() and np.isfinite(y).sum() == y.size - 64


# ------------------------------------------------------------------------------------------------ refusals
def fwd(**kw):
    a = dict(q=A, k=A, v=A, dt=1, B=1, H=4, Hkv=2, S=300, D=128, window=64, n_sink=4, scale=0.1, O=A, lse=A)
    a.update(kw)
    return lib.dfa_attn_fwd_sink(*(a[x] for x in ("q", "k", "v", "dt", "B", "H", "Hkv", "S", "D", "window", "n_sink", "scale",
                                                  "O", "lse")), None)


REFUSED = [
    (dict(D=96), dfa.DFA_ERR_UNSUPPORTED),
    (dict(dt=0), dfa.DFA_ERR_UNSUPPORTED),
    (dict(dt=7), dfa.DFA_ERR_INVALID_ARG),
    (dict(n_sink=129), dfa.DFA_ERR_UNSUPPORTED),
    (dict(n_sink=-1), dfa.DFA_ERR_INVALID_ARG),
    (dict(window=0), dfa.DFA_ERR_INVALID_ARG),
    (dict(window=-5), dfa.DFA_ERR_INVALID_ARG),
    (dict(H=3), dfa.DFA_ERR_INVALID_ARG),
    (dict(B=-1), dfa.DFA_ERR_INVALID_ARG),
    (dict(S=-1), dfa.DFA_ERR_INVALID_ARG),
    (dict(B=1 << 14, H=1 << 12, Hkv=1), dfa.DFA_ERR_INVALID_ARG),
    (dict(scale=float("nan")), dfa.DFA_ERR_INVALID_ARG),
    (dict(scale=-0.1), dfa.DFA_ERR_INVALID_ARG),
]


@pytest.mark.parametrize("kw,code", REFUSED + [(dict(O=MIS), dfa.DFA_ERR_INVALID_ARG), (dict(k=None), dfa.DFA_ERR_INVALID_ARG)])
def test_forward_refusals(kw, code):
    assert fwd(**kw) == code and dfa.dfa_last_error()


def bwd(**kw):
    a = dict(q=A, k=A, v=A, O=A, lse=A, dO=A, dt=1, B=1, H=4, Hkv=2, S=300, D=128, window=64, n_sink=4, scale=0.1, dQ=A,
             dK=A, dV=A, ws=A, n=1 << 40)
    a.update(kw)
    return lib.dfa_attn_bwd_sink(*(a[x] for x in ("q", "k", "v", "O", "lse", "dO", "dt", "B", "H", "Hkv", "S", "D", "window",
                                                  "n_sink", "scale", "dQ", "dK", "dV", "ws", "n")), None)


@pytest.mark.parametrize("kw,code", REFUSED + [
    (dict(dV=MIS), dfa.DFA_ERR_INVALID_ARG), (dict(dO=None), dfa.DFA_ERR_INVALID_ARG),
    (dict(ws=None), dfa.DFA_ERR_WORKSPACE), (dict(n=16), dfa.DFA_ERR_WORKSPACE), (dict(ws=MIS), dfa.DFA_ERR_INVALID_ARG),
    (dict(n=dfa.dfa_attn_bwd_sink_workspace_size(1, 4, 2, 300, 128, 64, 4) - 1), dfa.DFA_ERR_WORKSPACE)])
def test_backward_refusals(kw, code):
    assert bwd(**kw) == code and dfa.dfa_last_error()


def from_ckpt(**kw):
    a = dict(c=A, cn=1 << 40, lse=A, dO=A, dt=1, B=1, H=4, Hkv=2, S=300, D=128, window=64, n_sink=4, scale=0.1, dQ=A, dK=A,
             dV=A, ws=A, n=1 << 40)
    a.update(kw)
    return lib.dfa_attn_bwd_ckpt8(*(a[x] for x in ("c", "cn", "lse", "dO", "dt", "B", "H", "Hkv", "S", "D", "window", "n_sink",
                                                   "scale", "dQ", "dK", "dV", "ws", "n")), None)


@pytest.mark.parametrize("kw,code", REFUSED + [
    (dict(c=None), dfa.DFA_ERR_INVALID_ARG), (dict(c=MIS), dfa.DFA_ERR_INVALID_ARG),
    (dict(cn=dfa.dfa_ckpt8_size(1, 4, 2, 300, 128) - 1), dfa.DFA_ERR_INVALID_ARG),
    (dict(ws=None), dfa.DFA_ERR_WORKSPACE),
    (dict(n=dfa.dfa_attn_bwd_ckpt8_workspace_size(1, 4, 2, 300, 128, 64, 4) - 1), dfa.DFA_ERR_WORKSPACE)])
def test_checkpoint_backward_refusals(kw, code):
    assert from_ckpt(**kw) == code and dfa.dfa_last_error()


def test_checkpoint_refusals():
    n = dfa.dfa_ckpt8_size(2, 4, 2, 300, 64)
    q = 2 * 300 * 4 * 64
    assert q + q // 2 <= n <= 3 * q * (1 + 1 / 32) + 8 * 256
    ok = (A, A, A, A, 1, 2, 4, 2, 300, 64, A, n, None)
    for at, bad, code in ((0, None, 1), (3, MIS, 1), (4, 0, 2), (4, 9, 1), (9, 65, 2), (7, 3, 1), (10, None, 1), (11, n - 1, 1)):
        a = list(ok)
        a[at] = bad
        assert lib.dfa_ckpt8_save(*a) == code, (at, bad)
    ok = (A, n, 1, 2, 4, 2, 300, 64, A, A, A, A, None)
    for at, bad, code in ((0, MIS, 1), (1, n - 1, 1), (2, 0, 2), (7, 32, 2), (8, None, 1), (11, MIS, 1)):
        a = list(ok)
        a[at] = bad
        assert lib.dfa_ckpt8_restore(*a) == code, (at, bad)


def test_nothing_to_do_is_accepted_without_pointers():
    assert fwd(B=0, q=None, k=None, v=None, O=None, lse=None) == dfa.DFA_OK
    assert fwd(S=0, q=None, k=None, v=None, O=None, lse=None) == dfa.DFA_OK
    assert bwd(S=0, q=None, ws=None, n=0) == dfa.DFA_OK
    assert from_ckpt(B=0, c=None, cn=0, ws=None, n=0) == dfa.DFA_OK
    assert lib.dfa_ckpt8_save(None, None, None, None, 1, 1, 4, 2, 0, 64, None, 0, None) == dfa.DFA_OK


def test_size_queries_refuse_quietly():
    fwd(window=0)
    said = dfa.dfa_last_error()
    assert dfa.dfa_attn_bwd_sink_workspace_size(1, 4, 2, 300, 128, 0, 4) == 0
    assert dfa.dfa_attn_bwd_ckpt8_workspace_size(1, 4, 2, 300, 96, 8, 4) == 0
    assert dfa.dfa_ckpt8_size(1, 4, 3, 300, 128) == 0
    assert dfa.dfa_last_error() == said
    a, b = (dfa.dfa_attn_bwd_sink_workspace_size(1, 4, 2, 300, 128, 64, n) for n in (0, 4))
    assert 0 < a <= b


@pytest.mark.parametrize("n_sink", [0, 4])
@pytest.mark.parametrize("B,S", [(0, 300), (0, 0), (2, 0)])
def test_an_empty_batch_needs_no_workspace(B, S, n_sink):
    assert dfa.dfa_attn_bwd_sink_workspace_size(B, 4, 2, S, 128, 64, n_sink) == 0
    assert dfa.dfa_attn_bwd_ckpt8_workspace_size(B, 4, 2, S, 64, 64, n_sink) == 0


@pytest.mark.parametrize("n_sms", [1, 16, 152])
@pytest.mark.parametrize("B,H,Hkv,S,D,window,n_sink", [
    (1, 1, 1, 1, 64, 1, 1), (1, 8, 2, 1500, 128, 1500, 4), (2, 8, 4, 777, 64, 200, 8), (1, 32, 8, 32768, 128, 4096, 4),
    # more key tiles 0 than rounds were once looked at: 40000 of them, lists of one and of two tiles and longer
    (5000, 8, 8, 200, 128, 200, 4), (5000, 8, 8, 200, 128, 100, 4), (2400, 16, 16, 300, 128, 100, 4), (8000, 16, 8, 147, 64, 21, 128),
    (2071, 16, 2, 16205, 128, 14, 33), (6000, 16, 16, 129, 64, 1, 1),
])
def test_the_sinks_tile_always_has_ctas_of_its_own(B, H, Hkv, S, D, window, n_sink, n_sms):
    """The finer arithmetic of key tile 0 does not depend on how large the batch is."""
    p = dfa.dfa_debug_sink_bwd_plan(B, H, Hkv, S, D, window, n_sink, n_sms)
    assert p["rows"] == B * Hkv and p["items0"] >= p["rows"]
    assert 1 <= p["fine_ctas"] <= min(p["ctas"], p["items0"]) and p["ctas"] <= max(n_sms, 2)
    assert (p["ctas"] > p["fine_ctas"]) == (p["items"] > p["items0"])        # someone takes the others
    assert dfa.dfa_debug_sink_bwd_plan(B, H, Hkv, S, D, window, 0, n_sms)["fine_ctas"] == 0


def test_plan_refusals():
    plan = (ctypes.c_int32 * 8)()
    for bad in ((1, 4, 2, 300, 96, 64, 4, 152), (1, 4, 2, 300, 64, 0, 4, 152), (1, 4, 2, 300, 64, 64, 4, 0)):
        assert lib.dfa_debug_sink_bwd_plan(*bad, plan) != dfa.DFA_OK and dfa.dfa_last_error()
    assert lib.dfa_debug_sink_bwd_plan(1, 4, 2, 300, 64, 64, 4, 152, None) == dfa.DFA_ERR_INVALID_ARG


def test_the_binding_refuses_tensors_it_must_not_hand_on():
    t = lambda *s, dtype=torch.bfloat16: torch.zeros(s, dtype=dtype)  # noqa: E731
    q, k, lse = t(1, 8, 4, 64), t(1, 8, 2, 64), t(1, 4, 8, dtype=torch.float32)
    ck = t(1000, dtype=torch.uint8)
    for call in (lambda: dfa.dfa_attn_fwd_sink(q, k, k, 4), lambda: dfa.dfa_attn_bwd_sink(q, k, k, q, lse, q, 4),
                 lambda: dfa.dfa_ckpt8_save(q, k, k, q), lambda: dfa.dfa_ckpt8_restore(ck, 1, 4, 2, 8, 64),
                 lambda: dfa.dfa_attn_bwd_ckpt8(ck, lse, q, 2)):
        with pytest.raises(ValueError, match="CUDA"):
            call()
    for bad in ((q[0], k, k), (q, k, k[:, :4]), (q, k[:, :4], k[:, :4]), (q, t(1, 8, 2, 128), t(1, 8, 2, 128))):
        with pytest.raises(ValueError, match="must be"):
            dfa.dfa_attn_fwd_sink(*bad, 4)
    with pytest.raises(ValueError, match="dtype"):
        dfa.dfa_attn_fwd_sink(q, k, k.float(), 4)
    with pytest.raises(ValueError, match="contiguous"):
        dfa.dfa_attn_fwd_sink(q.transpose(1, 2).contiguous().transpose(1, 2), k, k, 4)


def decode(**kw):
    a = dict(q=A, k=A, v=A, dt=1, B=2, H=4, Hkv=2, S=300, D=128, ks=None, n=A, window=64, n_sink=4, scale=0.1, O=A, lse=A, ws=A,
             wn=1 << 40)
    a.update(kw)
    return lib.dfa_attn_decode_sink(*(a[x] for x in ("q", "k", "v", "dt", "B", "H", "Hkv", "S", "D", "ks", "n", "window",
                                                     "n_sink", "scale", "O", "lse", "ws", "wn")), None)


@pytest.mark.parametrize("kw,code", REFUSED + [
    (dict(S=0), dfa.DFA_ERR_INVALID_ARG), (dict(B=8193), dfa.DFA_ERR_UNSUPPORTED), (dict(n=None), dfa.DFA_ERR_INVALID_ARG),
    (dict(n=A + 2), dfa.DFA_ERR_INVALID_ARG), (dict(lse=None), dfa.DFA_ERR_INVALID_ARG), (dict(q=MIS), dfa.DFA_ERR_INVALID_ARG),
    (dict(ks=(ctypes.c_int64 * 3)(300 * 256, 256, 132)), dfa.DFA_ERR_INVALID_ARG),
    (dict(ks=(ctypes.c_int64 * 3)(300 * 256, -256, 128)), dfa.DFA_ERR_INVALID_ARG),
    (dict(ws=None), dfa.DFA_ERR_WORKSPACE), (dict(ws=MIS), dfa.DFA_ERR_INVALID_ARG),
    (dict(wn=dfa.dfa_attn_decode_sink_workspace_size(2, 4, 2, 128) - 1), dfa.DFA_ERR_WORKSPACE)])
def test_decode_refusals(kw, code):
    assert decode(**kw) == code and dfa.dfa_last_error()


@pytest.mark.parametrize("ks", [(0, 256, 128), (300 * 256, 0, 128), (300 * 256, 256, 0)])
def test_decode_refuses_broadcast_caches(ks):
    assert decode(ks=(ctypes.c_int64 * 3)(*ks)) == dfa.DFA_ERR_INVALID_ARG and "broadcast" in dfa.dfa_last_error()


def test_decode_of_no_sequence_and_size_queries():
    assert decode(B=0, q=None, k=None, v=None, n=None, ws=None, wn=0) == dfa.DFA_OK
    assert dfa.dfa_attn_decode_sink_workspace_size(8193, 4, 2, 128) == 0
    assert dfa.dfa_attn_decode_sink_workspace_size(1, 4, 2, 80) == 0
    assert dfa.dfa_attn_decode_sink_workspace_size(1, 4, 2, 128) > 0


def test_the_binding_refuses_decode_tensors():
    t = lambda *s, dtype=torch.bfloat16: torch.zeros(s, dtype=dtype)  # noqa: E731
    q, k, n = t(2, 4, 64), t(2, 8, 2, 64), t(2, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        dfa.dfa_attn_decode_sink(q, k, k, n, 4)
    for bad in ((q[:1], k, k), (q, k[0], k[0]), (q, k, t(2, 8, 2, 128)), (t(2, 4, 128), k, k)):
        with pytest.raises(ValueError, match="must be"):
            dfa.dfa_attn_decode_sink(*bad, n, 4)
    with pytest.raises(ValueError, match="strides"):
        dfa.dfa_attn_decode_sink(q, k, t(2, 2, 8, 64).transpose(1, 2), n, 4)
