"""The calls over a long cache on the CPU: the fp64 reference pinned by its
definitions and special cases, and what the calls refuse."""
import ctypes

import numpy as np
import pytest
import torch

from long_context_causal_gb300 import dfa
from oracle import cache, sink

lib = dfa.library()
A, MIS = 0x100000, 0x100004
FAR = [A + (i << 44) for i in range(16)]     # stand-in addresses far apart: validation fails before any use


def draw(B, S, H, Hkv, D, seed=0):
    r = np.random.default_rng(seed)
    return r.standard_normal((B, S, H, D)), r.standard_normal((B, S, Hkv, D)), r.standard_normal((B, S, Hkv, D))


# ------------------------------------------------------------------------------------------------ the reference
@pytest.mark.parametrize("window,n_sink", [(40, 0), (7, 0), (7, 3), (1, 0)])
def test_masses_are_column_sums_of_the_softmax(window, n_sink):
    q, k, v = draw(2, 40, 6, 2, 16)
    _, lse, _ = sink.attn_fwd(q, k, v, window, n_sink)
    got = cache.mass(q, k, lse, window, n_sink, 40)
    see = torch.from_numpy(sink.visible(40, window, n_sink))
    s = torch.einsum("bihd,bjhd->bhij", torch.from_numpy(q), torch.from_numpy(k).repeat_interleave(3, 2)) / 4
    p = torch.softmax(s.masked_fill(~see, -np.inf), -1)
    np.testing.assert_allclose(got, p.sum(2).reshape(2, 2, 3, 40).sum(2), atol=1e-12)
    np.testing.assert_allclose(got.sum(), 2 * 6 * 40)          # every query gives away one


def test_masses_are_gradients_of_the_log_sum():
    """d sum_i lse_i / d (an offset on key j's scores) is key j's mass."""
    q, k, v = draw(1, 12, 2, 1, 8, 1)
    _, lse, _ = sink.attn_fwd(q, k, v, 5, 2)
    m = cache.mass(q, k, lse, 5, 2, 4)
    see, h = sink.visible(12, 5, 2)[8:], 1e-6
    for j in range(12):
        d = []
        for e in (h, -h):
            s = np.einsum("ihd,jd->hij", q[0, 8:], k[0, :, 0]) * 8 ** -0.5 + e * (np.arange(12) == j)
            d.append(np.log((np.exp(s) * see).sum(-1)).sum())
        assert abs((d[0] - d[1]) / (2 * h) - m[0, 0, j]) < 1e-8


def test_a_steps_masses_are_the_last_querys():
    q, k, v = draw(2, 30, 4, 2, 16, 2)
    _, lse, _ = sink.attn_fwd(q, k, v, 9, 2)
    np.testing.assert_allclose(cache.step_mass(q[:, -1], k, [30, 30], 9, 2), cache.mass(q, k, lse, 9, 2, 1), atol=1e-12)


def test_what_is_kept():
    m = np.array([1.0, 5.0, 2.0, 5.0, 0.0, -0.0, np.nan, 3.0, 2.0, 9.0])
    assert cache.kept(m, 10, 12, 2, 2).tolist() == list(range(10))
    assert cache.kept(m, 10, 10, 0, 0).tolist() == list(range(10))
    assert cache.kept(m, 10, 3, 0, 0).tolist() == [1, 3, 9]
    assert cache.kept(m, 9, 3, 1, 1).tolist() == [0, 1, 8]
    assert cache.kept(m, 9, 5, 0, 0).tolist() == [1, 2, 3, 7, 8]
    assert cache.kept(m, 9, 7, 0, 0).tolist() == [0, 1, 2, 3, 4, 7, 8]     # of the zeros, the first
    assert cache.kept(m, 9, 8, 0, 0).tolist() == [0, 1, 2, 3, 4, 5, 7, 8]  # NaN last
    assert cache.kept(m, 10, 4, 2, 2).tolist() == [0, 1, 8, 9]


# ------------------------------------------------------------------------------------------------ refusals
def decode_mass(**kw):
    a = dict(q=FAR[0], k=FAR[1], v=FAR[2], dt=1, B=2, H=4, Hkv=2, S=300, D=128, ks=None, n=FAR[3], m=FAR[4], window=64, n_sink=4,
             scale=0.1, O=FAR[5], lse=FAR[6], mo=FAR[7], ws=FAR[8], wn=1 << 40)
    a.update(kw)
    return lib.dfa_attn_decode_mass(*(a[x] for x in ("q", "k", "v", "dt", "B", "H", "Hkv", "S", "D", "ks", "n", "m", "window",
                                                     "n_sink", "scale", "O", "lse", "mo", "ws", "wn")), None)


REFUSED = [(dict(dt=0), dfa.DFA_ERR_UNSUPPORTED), (dict(dt=5), dfa.DFA_ERR_INVALID_ARG), (dict(D=96), dfa.DFA_ERR_UNSUPPORTED),
           (dict(H=3), dfa.DFA_ERR_INVALID_ARG), (dict(B=-1), dfa.DFA_ERR_INVALID_ARG), (dict(scale=float("nan")), dfa.DFA_ERR_INVALID_ARG),
           (dict(scale=0.0), dfa.DFA_ERR_INVALID_ARG), (dict(window=0), dfa.DFA_ERR_INVALID_ARG), (dict(n_sink=-1), dfa.DFA_ERR_INVALID_ARG),
           (dict(n_sink=129), dfa.DFA_ERR_UNSUPPORTED)]


def mass(**kw):
    a = dict(q=FAR[0], k=FAR[1], lse=FAR[2], dt=1, B=2, H=4, Hkv=2, S=300, D=128, window=64, n_sink=4, n_last=300, scale=0.1, m=FAR[3],
             ws=FAR[4], wn=1 << 40)
    a.update(kw)
    return lib.dfa_attn_mass(*(a[x] for x in ("q", "k", "lse", "dt", "B", "H", "Hkv", "S", "D", "window", "n_sink", "n_last", "scale",
                                              "m", "ws", "wn")), None)


@pytest.mark.parametrize("kw,code", REFUSED + [
    (dict(S=-1), dfa.DFA_ERR_INVALID_ARG), (dict(n_last=0), dfa.DFA_ERR_INVALID_ARG), (dict(S=0, n_last=-3), dfa.DFA_ERR_INVALID_ARG),
    (dict(B=1 << 14, H=1 << 10, Hkv=1), dfa.DFA_ERR_INVALID_ARG), (dict(q=MIS), dfa.DFA_ERR_INVALID_ARG), (dict(k=None), dfa.DFA_ERR_INVALID_ARG),
    (dict(lse=A + 2), dfa.DFA_ERR_INVALID_ARG), (dict(m=None), dfa.DFA_ERR_INVALID_ARG), (dict(m=FAR[0]), dfa.DFA_ERR_INVALID_ARG),
    (dict(m=FAR[2] + 4), dfa.DFA_ERR_INVALID_ARG), (dict(ws=None), dfa.DFA_ERR_WORKSPACE), (dict(ws=MIS), dfa.DFA_ERR_INVALID_ARG),
    (dict(wn=dfa.dfa_attn_mass_workspace_size(2, 4, 2, 300, 128) - 1), dfa.DFA_ERR_WORKSPACE)])
def test_mass_refusals(kw, code):
    assert mass(**kw) == code and dfa.dfa_last_error()


def test_mass_of_nothing_and_size_queries():
    assert mass(B=0, q=None, k=None, lse=None, m=None, ws=None, wn=0) == dfa.DFA_OK
    assert mass(S=0, q=None, k=None, lse=None, m=None, ws=None, wn=0) == dfa.DFA_OK
    assert dfa.dfa_attn_mass_workspace_size(1, 4, 2, 300, 80) == 0 and dfa.dfa_attn_mass_workspace_size(1, 4, 3, 300, 64) == 0


@pytest.mark.parametrize("kw,code", REFUSED + [
    (dict(S=0), dfa.DFA_ERR_INVALID_ARG), (dict(B=8193), dfa.DFA_ERR_UNSUPPORTED), (dict(n=None), dfa.DFA_ERR_INVALID_ARG),
    (dict(mo=None), dfa.DFA_ERR_INVALID_ARG), (dict(m=A + 2), dfa.DFA_ERR_INVALID_ARG), (dict(mo=A + 1), dfa.DFA_ERR_INVALID_ARG),
    (dict(lse=None), dfa.DFA_ERR_INVALID_ARG), (dict(q=MIS), dfa.DFA_ERR_INVALID_ARG),
    (dict(ks=(ctypes.c_int64 * 3)(300 * 256, 256, 132)), dfa.DFA_ERR_INVALID_ARG),
    (dict(ks=(ctypes.c_int64 * 3)(0, 256, 128)), dfa.DFA_ERR_INVALID_ARG),
    (dict(mo=FAR[4] + 4), dfa.DFA_ERR_INVALID_ARG), (dict(mo=FAR[1] + 2 * 2 * 300 * 256 - 4), dfa.DFA_ERR_INVALID_ARG),
    (dict(mo=FAR[3] + 4), dfa.DFA_ERR_INVALID_ARG), (dict(ws=None), dfa.DFA_ERR_WORKSPACE), (dict(ws=MIS), dfa.DFA_ERR_INVALID_ARG),
    (dict(lse=FAR[7] + 4), dfa.DFA_ERR_INVALID_ARG), (dict(lse=FAR[7] + 4 * 2 * 2 * 300 - 4, m=None), dfa.DFA_ERR_INVALID_ARG),
    (dict(O=FAR[7]), dfa.DFA_ERR_INVALID_ARG), (dict(mo=FAR[5] + 2 * 2 * 4 * 128 - 4), dfa.DFA_ERR_INVALID_ARG),
    (dict(lse=FAR[5] + 8), dfa.DFA_ERR_INVALID_ARG), (dict(lse=FAR[4] + 8), dfa.DFA_ERR_INVALID_ARG), (dict(O=FAR[4] + 16), dfa.DFA_ERR_INVALID_ARG),
    (dict(wn=dfa.dfa_attn_decode_mass_workspace_size(2, 4, 2, 300, 128, 64, 4) - 1), dfa.DFA_ERR_WORKSPACE)])
def test_decode_mass_refusals(kw, code):
    assert decode_mass(**kw) == code and dfa.dfa_last_error()


def test_decode_mass_sizes():
    size = dfa.dfa_attn_decode_mass_workspace_size
    assert decode_mass(B=0, q=None, k=None, v=None, n=None, mo=None, ws=None, wn=0) == dfa.DFA_OK
    assert size(8193, 4, 2, 300, 128, 64, 4) == 0 and size(2, 4, 2, 300, 80, 64, 4) == 0 and size(2, 4, 2, 300, 128, 0, 4) == 0
    # the scores of the visible keys, in tiles of 64
    base = dfa.dfa_attn_decode_sink_workspace_size(2, 4, 2, 128)
    assert size(2, 4, 2, 300, 128, 300, 0) >= 4 * 2 * 4 * 300 and size(2, 4, 2, 300, 128, 1 << 30, 0) == size(2, 4, 2, 300, 128, 300, 9)
    assert size(2, 4, 2, 1 << 20, 128, 64, 4) <= base + 4 * 2 * 4 * 64 * 4 + 4096


def test_sizes_whose_tiles_32_bits_do_not_count():
    """A segment counts for two units more than its tiles: 2^30 of one tile are 3 * 2^30 units."""
    big = dict(B=8192, H=1 << 17, Hkv=1 << 17, S=64)
    assert dfa.dfa_attn_decode_mass_workspace_size(8192, 1 << 17, 1 << 17, 64, 128, 64, 0) == 0
    assert dfa.dfa_attn_decode_prefix_workspace_size(8192, 1 << 17, 1 << 17, 64, 128) == 0
    assert decode_mass(**big) == dfa.DFA_ERR_INVALID_ARG and prefix(**big) == dfa.DFA_ERR_INVALID_ARG


def prefix(**kw):
    a = dict(q=FAR[0], kp=FAR[1], vp=FAR[2], k=FAR[3], v=FAR[4], dt=1, B=2, H=4, Hkv=2, P=500, S=300, D=128, ps=None, ks=None, n=FAR[5],
             scale=0.1, O=FAR[6], lse=FAR[7], ws=FAR[8], wn=1 << 40)
    a.update(kw)
    return lib.dfa_attn_decode_prefix(*(a[x] for x in ("q", "kp", "vp", "k", "v", "dt", "B", "H", "Hkv", "P", "S", "D", "ps", "ks", "n",
                                                       "scale", "O", "lse", "ws", "wn")), None)


@pytest.mark.parametrize("kw,code", [r for r in REFUSED if "window" not in r[0] and "n_sink" not in r[0]] + [
    (dict(S=0), dfa.DFA_ERR_INVALID_ARG), (dict(P=-1), dfa.DFA_ERR_INVALID_ARG), (dict(P=(1 << 30) + 1), dfa.DFA_ERR_INVALID_ARG),
    (dict(B=8193), dfa.DFA_ERR_UNSUPPORTED), (dict(kp=None), dfa.DFA_ERR_INVALID_ARG), (dict(vp=MIS), dfa.DFA_ERR_INVALID_ARG),
    (dict(n=None), dfa.DFA_ERR_INVALID_ARG), (dict(lse=A + 2), dfa.DFA_ERR_INVALID_ARG), (dict(v=None), dfa.DFA_ERR_INVALID_ARG),
    (dict(ps=(ctypes.c_int64 * 2)(256, 12)), dfa.DFA_ERR_INVALID_ARG), (dict(ps=(ctypes.c_int64 * 2)(-256, 128)), dfa.DFA_ERR_INVALID_ARG),
    (dict(ps=(ctypes.c_int64 * 2)(0, 128)), dfa.DFA_ERR_INVALID_ARG), (dict(ps=(ctypes.c_int64 * 2)(256, 0)), dfa.DFA_ERR_INVALID_ARG),
    (dict(ks=(ctypes.c_int64 * 3)(0, 256, 128)), dfa.DFA_ERR_INVALID_ARG), (dict(ws=None), dfa.DFA_ERR_WORKSPACE),
    (dict(wn=dfa.dfa_attn_decode_prefix_workspace_size(2, 4, 2, 500, 128) - 1), dfa.DFA_ERR_WORKSPACE)])
def test_prefix_refusals(kw, code):
    assert prefix(**kw) == code and dfa.dfa_last_error()


def test_prefix_of_no_sequence_and_size_queries():
    size = dfa.dfa_attn_decode_prefix_workspace_size
    assert prefix(B=0, q=None, kp=None, vp=None, k=None, v=None, n=None, O=None, lse=None, ws=None, wn=0) == dfa.DFA_OK
    assert size(8193, 4, 2, 500, 128) == 0 and size(2, 4, 2, -1, 128) == 0 and size(2, 4, 2, 500, 96) == 0 and size(2, 4, 2, 0, 128) > 0


def evict(**kw):
    a = dict(k=FAR[0], v=FAR[1], dt=1, B=2, Hkv=3, S=300, D=128, ks=None, n=FAR[2], m=FAR[3], keep=40, first=2, recent=8, cap=64,
             os=None, ko=FAR[4], vo=FAR[5], lo=FAR[6], mo=FAR[7], kept=FAR[8])
    a.update(kw)
    return lib.dfa_cache_evict(*(a[x] for x in ("k", "v", "dt", "B", "Hkv", "S", "D", "ks", "n", "m", "keep", "first", "recent", "cap",
                                                "os", "ko", "vo", "lo", "mo", "kept")), None)


def s3(*x):
    return (ctypes.c_int64 * 3)(*x)


CACHE = 2 * 2 * 300 * 3 * 128        # bytes of k


@pytest.mark.parametrize("kw,code", [
    (dict(dt=5), dfa.DFA_ERR_INVALID_ARG), (dict(D=96), dfa.DFA_ERR_UNSUPPORTED), (dict(B=-1), dfa.DFA_ERR_INVALID_ARG),
    (dict(Hkv=0), dfa.DFA_ERR_INVALID_ARG), (dict(S=0), dfa.DFA_ERR_INVALID_ARG), (dict(keep=0), dfa.DFA_ERR_INVALID_ARG),
    (dict(first=-1), dfa.DFA_ERR_INVALID_ARG), (dict(recent=-1), dfa.DFA_ERR_INVALID_ARG), (dict(first=33), dfa.DFA_ERR_INVALID_ARG),
    (dict(first=1 << 30, recent=1 << 30, keep=1 << 30, cap=1 << 30), dfa.DFA_ERR_INVALID_ARG),
    (dict(cap=39), dfa.DFA_ERR_INVALID_ARG), (dict(S=1 << 30, keep=1 << 30, cap=1 << 30, Hkv=1 << 10), dfa.DFA_ERR_INVALID_ARG),
    (dict(ks=s3(300 * 384, 384, 132)), dfa.DFA_ERR_INVALID_ARG), (dict(os=s3(64 * 384, -384, 128)), dfa.DFA_ERR_INVALID_ARG),
    (dict(os=s3(0, 384, 128)), dfa.DFA_ERR_INVALID_ARG), (dict(os=s3(64 * 384, 0, 128)), dfa.DFA_ERR_INVALID_ARG),
    (dict(k=MIS), dfa.DFA_ERR_INVALID_ARG), (dict(vo=None), dfa.DFA_ERR_INVALID_ARG), (dict(kept=None), dfa.DFA_ERR_INVALID_ARG),
    (dict(lo=A + 2), dfa.DFA_ERR_INVALID_ARG), (dict(m=None), dfa.DFA_ERR_INVALID_ARG), (dict(vo=FAR[4]), dfa.DFA_ERR_INVALID_ARG),
    (dict(ko=FAR[0]), dfa.DFA_ERR_INVALID_ARG), (dict(vo=FAR[0] + CACHE - 16), dfa.DFA_ERR_INVALID_ARG),
    (dict(lo=FAR[2]), dfa.DFA_ERR_INVALID_ARG), (dict(mo=FAR[3]), dfa.DFA_ERR_INVALID_ARG), (dict(kept=FAR[3]), dfa.DFA_ERR_INVALID_ARG),
    # outputs among each other: small ones; slices of one buffer a row, a head, a few elements or a sequence apart
    (dict(kept=FAR[7] + 8), dfa.DFA_ERR_INVALID_ARG), (dict(lo=FAR[8] + 4 * 2 * 3 * 40 - 4), dfa.DFA_ERR_INVALID_ARG), (dict(lo=FAR[7]), dfa.DFA_ERR_INVALID_ARG),
    (dict(mo=FAR[4]), dfa.DFA_ERR_INVALID_ARG), (dict(kept=FAR[5] + 64), dfa.DFA_ERR_INVALID_ARG), (dict(lo=FAR[5] + 4), dfa.DFA_ERR_INVALID_ARG),
    *[(dict(vo=FAR[4] + 2 * d), dfa.DFA_ERR_INVALID_ARG) for d in (8, 128, 384, 10 * 384, 64 * 384)],
    *[(dict(ko=FAR[5] + 2 * d, vo=FAR[5], os=s3(130 * 400, 400, 128)), dfa.DFA_ERR_INVALID_ARG) for d in (16, 120, 63 * 400, 130 * 400 + 63 * 400 + 256 + 120)],
    (dict(vo=FAR[4] + 2 * 3 * 800, os=s3(64 * 400, 400, 128), B=1, cap=128), dfa.DFA_ERR_INVALID_ARG),
    (dict(vo=FAR[4] + 2 * (1 << 16), os=s3(8, 8, 8), Hkv=64, cap=1 << 20, S=64, B=64), dfa.DFA_ERR_INVALID_ARG),
])
def test_evict_refusals(kw, code):
    assert evict(**kw) == code and dfa.dfa_last_error()


def test_evict_of_no_sequence():
    assert evict(B=0, k=None, v=None, n=None, m=None, ko=None, vo=None, lo=None, mo=None, kept=None) == dfa.DFA_OK


def test_the_binding_refuses_cache_tensors():
    t = lambda *s, dtype=torch.bfloat16: torch.zeros(s, dtype=dtype)  # noqa: E731
    q, k, n, m = t(2, 4, 64), t(2, 8, 2, 64), t(2, dtype=torch.int32), t(2, 2, 8, dtype=torch.float32)
    for call in (lambda: dfa.dfa_attn_decode_mass(q, k, k, n), lambda: dfa.dfa_cache_evict(k, k, n, m, 4)):
        with pytest.raises(ValueError, match="CUDA"):
            call()
    lse = t(2, 4, 8, dtype=torch.float32)
    with pytest.raises(ValueError, match="CUDA"):
        dfa.dfa_attn_mass(t(2, 8, 4, 64), k, lse)
    for bad in ((q, k), (t(2, 8, 4, 64), k[:, :4]), (t(2, 8, 4, 128), k)):
        with pytest.raises(ValueError, match="must be"):
            dfa.dfa_attn_mass(*bad, lse)
    for bad in ((q[:1], k, k), (q, k[0], k[0]), (q, k, t(2, 8, 2, 128)), (t(2, 4, 128), k, k)):
        with pytest.raises(ValueError, match="must be"):
            dfa.dfa_attn_decode_mass(*bad, n)
    kp = t(9, 2, 64)
    with pytest.raises(ValueError, match="CUDA"):
        dfa.dfa_attn_decode_prefix(q, kp, kp, k, k, n)
    for bad in ((kp[0], kp[0]), (kp, kp[:4]), (kp[:, :1], kp[:, :1]), (t(9, 2, 128), t(9, 2, 128)), (kp.float(), kp.float()),
                (kp, t(2, 9, 64).transpose(0, 1))):
        with pytest.raises(ValueError, match="must"):
            dfa.dfa_attn_decode_prefix(q, *bad, k, k, n)
    for other in (t(2, 8, 2, 128), k.float(), t(2, 2, 8, 64).transpose(1, 2)):
        with pytest.raises(ValueError, match="must"):
            dfa.dfa_cache_evict(k, other, n, m, 4)
    with pytest.raises(TypeError, match="dtype"):
        dfa.dfa_cache_evict(k.half(), k.half(), n, m, 4)
