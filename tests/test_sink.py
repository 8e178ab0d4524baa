"""Windowed attention with sinks and the 8-bit checkpoints on the GPU, against
the fp64 reference (oracle/sink.py).

Tolerances are sums over the terms of each element.  With u = 2^-8, half a
step of bf16 relative to the value:
  O    the probabilities are rounded once (u times the sum of P |v|) and the
       result once (u |O|);
  dV   likewise (P and the result);
  dQ, dK  P and dS are rounded (2 u times the sum of |dS| |k| or |dS| |q|),
       the result once;
  P of dS is kept in fp16 times 2^14 (2^8 from a checkpoint): 11 bits, more
       than the above counts, but for P below 2^-28 (2^-22), where it is off by
       up to half the smallest fp16 number, 2^-25 / 2^14 = 2^-39 (2^-33);
and fp32 sums of up to D = 128 products move a score by less than 2^-13 and
dO.v - Delta by less than 2^-16 of the magnitudes it is the difference of.
"""
import numpy as np
import pytest
import torch

from long_context_causal_gb300 import dfa
from long_context_causal_gb300.inputs import make
from oracle import sink

pytestmark = pytest.mark.gpu
DEV = "cuda"
U, F, F2 = 2.0 ** -8, 2.0 ** -12, 2.0 ** -16


def np64(t):
    return t.detach().double().cpu().numpy()


def close(got, ref, tol, what):
    bad = ~(np.abs(np64(got) - ref) <= tol)
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size}, first at {np.argwhere(bad)[0]}, worst {np.nanmax(np.abs(np64(got) - ref) / (tol + 1e-30)):.3g} of the tolerance"


def check_fwd(O, lse, q, k, v, window, n_sink, scale=None):
    Or, lr, size = sink.attn_fwd(np64(q), np64(k), np64(v), window, n_sink, scale)
    close(O, Or, (U + F) * size + U * np.abs(Or), "O")
    close(lse, lr, 2 * F, "lse")


def check_bwd(grads, q, k, v, O, lse, do, window, n_sink, scale=None, least=2.0 ** -39):
    ref = sink.attn_bwd(*(np64(t) for t in (q, k, v, O, lse, do)), window, n_sink, scale)
    for got, name in zip(grads, ("dQ", "dK", "dV")):
        r, terms, cancel, floor = ref[name]
        close(got, r, ((1 if name == "dV" else 2) * U + F) * terms + F2 * cancel + least * floor + U * np.abs(r) + 1e-30, name)


# (B, H, Hkv, S, D, window, n_sink)
CASES = [
    (1, 1, 1, 1, 128, 1, 0), (2, 2, 1, 1, 64, 5, 3),
    (1, 2, 1, 2, 128, 1, 1), (1, 2, 2, 127, 128, 16, 2), (1, 2, 2, 128, 64, 128, 128),
    (2, 4, 2, 129, 64, 32, 1), (1, 4, 1, 255, 128, 100, 0), (1, 3, 3, 256, 128, 128, 16),
    (2, 2, 1, 257, 128, 129, 17), (1, 8, 2, 300, 64, 1, 4), (1, 2, 2, 385, 128, 127, 128),
    (1, 2, 1, 640, 128, 256, 33), (1, 6, 2, 1000, 128, 200, 8), (1, 2, 2, 1000, 64, 1000, 4),
    (1, 2, 1, 1500, 128, 2000, 0), (3, 2, 2, 513, 64, 130, 127),
    (1, 4, 2, 2500, 128, 100, 4), (1, 2, 1, 4200, 64, 257, 128), (1, 2, 2, 3100, 128, 1, 1),
]
IDS = ["B{}H{}kv{}S{}D{}w{}s{}".format(*c) for c in CASES]


@pytest.mark.parametrize("case", CASES, ids=IDS)
def test_forward(case):
    B, H, Hkv, S, D, window, n_sink = case
    q, k, v, _ = make(B, H, Hkv, S, D, torch.bfloat16, device=DEV, seed=31)
    O, lse = dfa.dfa_attn_fwd_sink(q, k, v, window, n_sink)
    dfa.dfa_check_errors()
    check_fwd(O, lse, q, k, v, window, n_sink)


@pytest.mark.parametrize("case", CASES, ids=IDS)
def test_backward(case):
    B, H, Hkv, S, D, window, n_sink = case
    q, k, v, do = make(B, H, Hkv, S, D, torch.bfloat16, device=DEV, seed=32)
    O, lse = dfa.dfa_attn_fwd_sink(q, k, v, window, n_sink)
    grads = dfa.dfa_attn_bwd_sink(q, k, v, O, lse, do, window, n_sink)
    dfa.dfa_check_errors()
    check_bwd(grads, q, k, v, O, lse, do, window, n_sink)


def rows_fwd(q, k, v, window, n_sink):
    """O, lse and sum_j p_j |v_j| in 64 bits, rows in blocks that read only the keys they can see."""
    B, S, H, D = q.shape
    out = [torch.empty(B, S, H, D, dtype=torch.float64, device=q.device) for _ in range(2)]
    lse = torch.empty(B, H, S, dtype=torch.float64, device=q.device)
    for a in range(0, S, 1024):
        b = min(a + 1024, S)
        lo = max(a - window + 1, 0)
        cols = torch.cat([torch.arange(0, min(n_sink, lo), device=q.device), torch.arange(lo, b, device=q.device)])
        rows = torch.arange(a, b, device=q.device)[:, None]
        see = (cols <= rows) & ((cols > rows - window) | (cols < n_sink))
        for h in range(H):
            kh, vh = (t[:, cols, h * k.shape[2] // H].double() for t in (k, v))
            s = (q[:, a:b, h].double() @ kh.transpose(1, 2) * D ** -0.5).masked_fill(~see, float("-inf"))
            lse[:, h, a:b] = torch.logsumexp(s, -1)
            p = torch.exp(s - lse[:, h, a:b, None])
            out[0][:, a:b, h], out[1][:, a:b, h] = p @ vh, p @ vh.abs()
    return out[0], lse, out[1]


# Few blocks, or a last round that is not full: blocks whose key lists several CTAs share, in pieces that hold no key
# of a query tile, the sinks alone, or nothing; query tiles past the end; whole blocks before shared ones.
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("B,H,Hkv,S,window,n_sink", [
    (1, 1, 1, 1100, 2000, 0), (1, 1, 1, 2000, 2000, 0), (1, 1, 1, 3001, 2500, 128), (2, 3, 3, 1111, 900, 17),
    (1, 8, 2, 1500, 1500, 0), (1, 2, 1, 2200, 1400, 5), (1, 8, 4, 2300, 1500, 33), (1, 2, 2, 2817, 2817, 0),
    (1, 8, 2, 4000, 4000, 0), (1, 4, 2, 12000, 2000, 1), (1, 1, 1, 20000, 700, 128),
])
def test_blocks_shared_by_several_ctas(B, H, Hkv, S, window, n_sink, D):
    q, k, v, _ = make(B, H, Hkv, S, D, torch.bfloat16, device=DEV, seed=71)
    k[:, :200] *= 3                       # the pieces' maxima differ
    O, lse = dfa.dfa_attn_fwd_sink(q, k, v, window, n_sink)
    again = dfa.dfa_attn_fwd_sink(q, k, v, window, n_sink)
    dfa.dfa_check_errors()
    Or, lr, size = rows_fwd(q, k, v, window, n_sink)
    close(O, np64(Or), (U + F) * np64(size) + U * np.abs(np64(Or)), "O")
    close(lse, np64(lr), 2 * F, "lse")
    assert torch.equal(O, again[0]) and torch.equal(lse, again[1])


def test_sharp_scores_rescale():
    """Maxima that rise by more than 2^8 along the keys, and sinks above all of them."""
    q, k, v, do = make(1, 2, 1, 900, 128, torch.bfloat16, device=DEV, seed=33, k_scale=4.0)
    k[:, :4] *= 3
    k[:, 400:] *= 2
    O, lse = dfa.dfa_attn_fwd_sink(q, k, v, 300, 4, scale=0.2)
    grads = dfa.dfa_attn_bwd_sink(q, k, v, O, lse, do, 300, 4, scale=0.2)
    dfa.dfa_check_errors()
    # scores reach 200: fp32 moves them by 2^-24 * 200 * a few, far below F
    check_fwd(O, lse, q, k, v, 300, 4, 0.2)
    check_bwd(grads, q, k, v, O, lse, do, 300, 4, 0.2)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("S,window,n_sink", [(900, 40, 128), (300, 1000, 100)])
def test_sinks_that_share_a_direction(D, S, window, n_sink):
    """A row's dS sum to nearly zero, so what all keys share cancels in dQ: the
    roundings of key tile 0's dS must not bring it back.  There P is rounded to
    fp16 (half a step: 2^-11) and dS held in two bf16 numbers (2^-8 squared);
    the other tiles round dS to bf16."""
    B, H, Hkv = 1, 4, 2
    q, k, v, do = make(B, H, Hkv, S, D, torch.bfloat16, device=DEV, seed=36)
    u = torch.randn(Hkv, D, device=DEV, generator=torch.Generator(DEV).manual_seed(37))
    q += (0.25 * u.repeat_interleave(H // Hkv, 0)).bfloat16()
    k[:, :n_sink] = (0.1 * k[:, :n_sink] + 3 * u).bfloat16()
    O, lse = dfa.dfa_attn_fwd_sink(q, k, v, window, n_sink)
    dQ, dK, dV = dfa.dfa_attn_bwd_sink(q, k, v, O, lse, do, window, n_sink)
    dfa.dfa_check_errors()
    args = [np64(t) for t in (q, k, v, O, lse, do)]
    r, terms, cancel, floor = sink.attn_bwd(*args, window, n_sink)["dQ"]
    # what key tile 0 adds to the terms
    first = np.zeros_like(r)
    see = sink.visible(S, window, n_sink)
    for h in range(H):
        g = h // (H // Hkv)
        qh, kh, vh, oh, dh = (np64(t)[0] for t in (q[:, :, h], k[:, :, g], v[:, :, g], O[:, :, h], do[:, :, h]))
        p = np.where(see, np.exp(D ** -0.5 * qh @ kh.T - np64(lse)[0, h][:, None]), 0)
        ds = np.abs(p * (dh @ vh.T - (dh * oh).sum(1, keepdims=True))) * D ** -0.5
        first[0, :, h] = ds[:, :128] @ np.abs(kh[:128])
    close(dQ, r, (2.0 ** -11 + 2.0 ** -16) * first + U * (terms - first) + F * terms + F2 * cancel + 2.0 ** -39 * floor
          + U * np.abs(r) + 1e-30, "dQ")
    check_bwd((dQ, dK, dV), q, k, v, O, lse, do, window, n_sink)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("S,window", [(6, 100), (40, 100), (200, 30)])
def test_dv_of_the_sinks_tile(D, S, window):
    """The keys of tile 0 of a problem with sinks: their dV sums over the most queries, and P comes to it in two
    bf16 numbers (2^-8 squared), so that an element whose terms cancel is not off by their rounding."""
    B, H, Hkv, n_sink = 2, 4, 2, 1
    q, k, v, do = make(B, H, Hkv, S, D, torch.bfloat16, device=DEV, seed=38)
    u = torch.randn(Hkv, D, device=DEV, generator=torch.Generator(DEV).manual_seed(39))
    q += (0.25 * u.repeat_interleave(H // Hkv, 0)).bfloat16()
    k[:, :n_sink] = (0.3 * k[:, :n_sink] + 1.5 * u).bfloat16()
    O, lse = dfa.dfa_attn_fwd_sink(q, k, v, window, n_sink)
    dV = dfa.dfa_attn_bwd_sink(q, k, v, O, lse, do, window, n_sink)[2]
    dfa.dfa_check_errors()
    r, terms, cancel, floor = sink.attn_bwd(*(np64(t) for t in (q, k, v, O, lse, do)), window, n_sink)["dV"]
    tol = (2.0 ** -16 + F) * terms + F2 * cancel + 2.0 ** -39 * floor + U * np.abs(r) + 1e-30
    close(dV[:, :128], r[:, :128], tol[:, :128], "dV")


def test_dv_of_the_sinks_tile_in_a_large_batch():
    """As above with more lists of key tile 0 (40000) than 256 rounds of CTAs take: the arithmetic is the same."""
    B, H, Hkv, S, D, window, n_sink = 5000, 8, 8, 130, 64, 100, 1
    q, k, v, do = make(B, H, Hkv, S, D, torch.bfloat16, device=DEV, seed=38)
    u = torch.randn(Hkv, D, device=DEV, generator=torch.Generator(DEV).manual_seed(39))
    q += (0.25 * u).bfloat16()
    k[:, :n_sink] = (0.3 * k[:, :n_sink] + 1.5 * u).bfloat16()
    O, lse = dfa.dfa_attn_fwd_sink(q, k, v, window, n_sink)
    dQ, dK, dV = dfa.dfa_attn_bwd_sink(q, k, v, O, lse, do, window, n_sink)
    dfa.dfa_check_errors()
    some = [0, 1, 2499, 4999]
    args = [t[some] for t in (q, k, v, O, lse, do)]
    check_bwd([t[some] for t in (dQ, dK, dV)], *args, window, n_sink)
    r, terms, cancel, floor = sink.attn_bwd(*(np64(t) for t in args), window, n_sink)["dV"]
    tol = (2.0 ** -16 + F) * terms + F2 * cancel + 2.0 ** -39 * floor + U * np.abs(r) + 1e-30
    close(dV[some][:, :128], r[:, :128], tol[:, :128], "dV")


def test_window_over_every_key_is_the_causal_call():
    q, k, v, do = make(2, 4, 2, 700, 128, torch.bfloat16, device=DEV, seed=34)
    O, lse = dfa.dfa_attn_fwd_sink(q, k, v, 700, 9)
    O2, lse2 = dfa.dfa_attn_fwd(q, k, v)
    torch.testing.assert_close(O.float(), O2.float(), rtol=2 * U, atol=1e-4)
    torch.testing.assert_close(lse, lse2, rtol=0, atol=1e-5)
    for a, b in zip(dfa.dfa_attn_bwd_sink(q, k, v, O2, lse2, do, 1 << 30), dfa.dfa_attn_bwd(q, k, v, O2, lse2, do)):
        err = (a.float() - b.float()).norm() / b.float().norm()
        assert err <= 3 * U, err     # each side rounds P, dS and the result; far from their worst at once


@pytest.mark.parametrize("D", [64, 128])
def test_bits_repeat_and_neighbours_stay(D):
    """O, lse, dK, dV have the same bits on every call, and nothing is written
    outside the outputs (sequences of a batch end inside a tile)."""
    B, H, Hkv, S, W, N = 3, 4, 2, 1337, 90, 5
    q, k, v, do = make(B, H, Hkv, S, D, torch.bfloat16, device=DEV, seed=35)
    def framed(shape, dtype):
        n = int(np.prod(shape))
        buf = torch.full((n + 8192,), 7.0, dtype=dtype, device=DEV)
        return buf, buf[4096:4096 + n].view(shape)
    runs = []
    for _ in range(3):
        bufs = [framed(q.shape, q.dtype), framed((B, H, S), torch.float32)]
        dfa.dfa_attn_fwd_sink(q, k, v, W, N, O=bufs[0][1], lse=bufs[1][1])
        bufs += [framed(q.shape, q.dtype), framed(k.shape, q.dtype), framed(k.shape, q.dtype)]
        nb = dfa.dfa_attn_bwd_sink_workspace_size(B, H, Hkv, S, D, W, N)
        ws = torch.full((nb + 4096,), 0xAB, dtype=torch.uint8, device=DEV)   # dirty, with a frame behind
        dfa.dfa_attn_bwd_sink(q, k, v, bufs[0][1], bufs[1][1], do, W, N, dQ=bufs[2][1], dK=bufs[3][1], dV=bufs[4][1],
                              workspace_buf=ws[:nb])
        assert (ws[nb:] == 0xAB).all()
        for buf, t in bufs:
            n = t.numel()
            assert (buf[:4096] == 7).all() and (buf[4096 + n:] == 7).all()
        runs.append([t.clone() for _, t in bufs])
    dfa.dfa_check_errors()
    for r in runs[1:]:
        for z in (0, 1, 3, 4):
            assert torch.equal(r[z], runs[0][z])
        torch.testing.assert_close(r[2].float(), runs[0][2].float(), rtol=2 * U, atol=1e-3)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("S,window", [(3, 100), (6, 100), (40, 100), (200, 30), (1500, 2000)])
def test_dk_of_the_sinks_tile(D, S, window):
    """The same for dK, whose terms are dS q: P of dS is rounded to fp16 (half a step: 2^-11) and dS held in two bf16
    numbers."""
    B, H, Hkv, n_sink = 2, 4, 2, 1
    q, k, v, do = make(B, H, Hkv, S, D, torch.bfloat16, device=DEV, seed=38)
    u = torch.randn(Hkv, D, device=DEV, generator=torch.Generator(DEV).manual_seed(39))
    q += (0.25 * u.repeat_interleave(H // Hkv, 0)).bfloat16()
    k[:, :n_sink] = (0.3 * k[:, :n_sink] + 1.5 * u).bfloat16()
    O, lse = dfa.dfa_attn_fwd_sink(q, k, v, window, n_sink)
    dK = dfa.dfa_attn_bwd_sink(q, k, v, O, lse, do, window, n_sink)[1]
    dfa.dfa_check_errors()
    r, terms, cancel, floor = sink.attn_bwd(*(np64(t) for t in (q, k, v, O, lse, do)), window, n_sink)["dK"]
    tol = (2.0 ** -11 + 2.0 ** -16 + F) * terms + F2 * cancel + 2.0 ** -39 * floor + U * np.abs(r) + 1e-30
    close(dK[:, :128], r[:, :128], tol[:, :128], "dK")


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("n_sink", [0, 4])
@pytest.mark.parametrize("down", [np.log(3), np.log(8), np.log(2000)])
def test_where_p_saturates(D, n_sink, down):
    """An lse lower than the forward's, as the call says it: dQ and dK take P as 65504 / 2^14 at most (from a
    checkpoint 65504 / 2^8), dV as it is."""
    B, H, Hkv, S, window = 1, 4, 2, 300, 70
    q, k, v, do = make(B, H, Hkv, S, D, torch.bfloat16, device=DEV, seed=46)
    O, lse = dfa.dfa_attn_fwd_sink(q, k, v, window, n_sink)
    lse[:, :, 10:200:3] -= down
    args = [np64(t) for t in (q, k, v, O)]
    for grads, args, shift in (
            (dfa.dfa_attn_bwd_sink(q, k, v, O, lse, do, window, n_sink), args, 14),
            (dfa.dfa_attn_bwd_ckpt8(dfa.dfa_ckpt8_save(q, k, v, O), lse, do, Hkv, window, n_sink), [sink.ckpt8(t) for t in args], 8)):
        ref = sink.attn_bwd(*args, np64(lse), np64(do), window, n_sink, most=65504 / 2 ** shift)
        for got, name in zip(grads, ("dQ", "dK", "dV")):
            r, terms, cancel, floor = ref[name]
            close(got, r, ((1 if name == "dV" else 2) * U + F) * terms + F2 * cancel + 2.0 ** (-25 - shift) * floor
                  + U * np.abs(r) + 1e-30, name)
    dfa.dfa_check_errors()


# ------------------------------------------------------------------------------------------------ checkpoints
@pytest.mark.parametrize("B,H,Hkv,S,D", [(1, 1, 1, 1, 64), (1, 3, 1, 1, 128), (2, 4, 2, 129, 128), (1, 8, 8, 501, 64),
                                         (3, 6, 3, 77, 128)])
def test_checkpoint_holds_the_definitions_values(B, H, Hkv, S, D):
    q, k, v, o = make(B, H, Hkv, S, D, torch.bfloat16, device=DEV, seed=41)
    q *= 10.0 ** torch.randint(-20, 20, (B, S, H, 1), device=DEV, generator=torch.Generator(DEV).manual_seed(1)).float()
    k[:, 0, 0, :32] = 0
    v[:, S // 2, 0, 32:40] = 2.0 ** -126       # beside larger elements, and alone with the smallest exponent
    v[:, -1, -1, 32:] = 2.0 ** -124
    o[:, 0, 0, 3] = -3.3e38
    ckpt = dfa.dfa_ckpt8_save(q, k, v, o)
    assert ckpt.numel() == dfa.dfa_ckpt8_size(B, H, Hkv, S, D)
    for got, t, name in zip(dfa.dfa_ckpt8_restore(ckpt, B, H, Hkv, S, D), (q, k, v, o), "qkvO"):
        assert got.dtype == torch.bfloat16 and np.array_equal(np64(got), sink.ckpt8(np64(t))), name


def test_checkpoint_of_non_finite_groups():
    q, k, v, o = make(1, 2, 1, 40, 64, torch.bfloat16, device=DEV, seed=42)
    q[0, 3, 1, 40], k[0, 5, 0, 0], o[0, 39, 1, 63] = float("inf"), float("nan"), float("-inf")
    back = dfa.dfa_ckpt8_restore(dfa.dfa_ckpt8_save(q, k, v, o), 1, 2, 1, 40, 64)
    for got, t in zip(back, (q, k, v, o)):
        assert np.array_equal(np64(got), sink.ckpt8(np64(t)), equal_nan=True)
    assert sum(int(t.isnan().sum()) for t in back) == 96


def test_checkpoint_stays_inside_its_buffer():
    B, H, Hkv, S, D = 1, 3, 1, 33, 64
    q, k, v, o = make(B, H, Hkv, S, D, torch.bfloat16, device=DEV, seed=43)
    n = dfa.dfa_ckpt8_size(B, H, Hkv, S, D)
    buf = torch.full((n + 512,), 0x5A, dtype=torch.uint8, device=DEV)
    a = dfa.dfa_ckpt8_save(q, k, v, o, ckpt=buf[256:256 + n])
    assert (buf[:256] == 0x5A).all() and (buf[256 + n:] == 0x5A).all()
    b = dfa.dfa_ckpt8_save(q, k, v, o)
    for x, y in zip(dfa.dfa_ckpt8_restore(a, B, H, Hkv, S, D), dfa.dfa_ckpt8_restore(b, B, H, Hkv, S, D)):
        assert torch.equal(x, y)


@pytest.mark.parametrize("case", [c for c in CASES if c[3] in (1, 129, 257, 300, 640, 1000, 1500, 2500, 3100)],
                         ids=lambda c: "B{}H{}kv{}S{}D{}w{}s{}".format(*c))
def test_backward_from_a_checkpoint(case):
    """The training step: forward, save, and the backward from what was saved."""
    B, H, Hkv, S, D, window, n_sink = case
    q, k, v, do = make(B, H, Hkv, S, D, torch.bfloat16, device=DEV, seed=44)
    O, lse = dfa.dfa_attn_fwd_sink(q, k, v, window, n_sink)
    ckpt = dfa.dfa_ckpt8_save(q, k, v, O)
    held = [torch.from_numpy(sink.ckpt8(np64(t))).to(DEV) for t in (q, k, v, O)]
    del q, k, v, O
    n_fwd = dfa.dfa_launch_count("fwd")
    grads = dfa.dfa_attn_bwd_ckpt8(ckpt, lse, do, Hkv, window, n_sink)
    dfa.dfa_check_errors()
    assert dfa.dfa_launch_count("fwd") == n_fwd
    check_bwd(grads, *held, lse, do, window, n_sink, least=2.0 ** -33)


def test_causal_backward_from_a_checkpoint():
    """Without a window it is the backward of dfa_attn_fwd, from rounded tensors."""
    q, k, v, do = make(1, 4, 1, 770, 128, torch.bfloat16, device=DEV, seed=45)
    O, lse = dfa.dfa_attn_fwd(q, k, v)
    grads = dfa.dfa_attn_bwd_ckpt8(dfa.dfa_ckpt8_save(q, k, v, O), lse, do, 1)
    dfa.dfa_check_errors()
    held = [sink.ckpt8(np64(t)) for t in (q, k, v, O)]
    check_bwd(grads, *(torch.from_numpy(t) for t in held), lse, do, 770, 0, least=2.0 ** -33)
    # and the checkpoint's own rounding, 2^-7 of a group's largest at most, moves the gradients little
    for a, b in zip(grads, dfa.dfa_attn_bwd(q, k, v, O, lse, do)):
        assert (a.float() - b.float()).norm() <= 0.05 * b.float().norm()


# ------------------------------------------------------------------------------------------------ single tokens
# (B, H, Hkv, S_max, D, window, n_sink, lengths)
DECODE = [
    (1, 1, 1, 1, 64, 1, 0, [1]),
    (1, 4, 1, 64, 128, 64, 4, [64]),
    (3, 4, 2, 100, 128, 1, 1, [0, 1, 100]),
    (2, 8, 8, 300, 64, 65, 3, [66, 300]),
    (4, 6, 2, 1000, 128, 128, 128, [129, 256, 257, 1000]),
    (5, 40, 2, 700, 64, 200, 17, [0, 0, 17, 217, 700]),          # 20 heads to a key/value head: two blocks of 16
    (2, 33, 1, 500, 128, 1000, 5, [499, 1]),
    (1, 8, 2, 5000, 128, 5000, 4, [4999]),
    (1, 2, 1, 9000, 64, 3000, 100, [9000]),
    (17, 4, 4, 260, 128, 70, 4, [0] * 8 + [260, 3, 70, 71, 74, 75, 138, 139, 200]),
    (300, 2, 1, 40, 64, 16, 2, [i % 41 for i in range(300)]),
    (2, 32, 2, 600, 128, 500, 3, [599, 0]),                       # 16 heads to a key/value head
    (1, 16, 8, 4096, 128, 4096, 0, [4096]), (1, 16, 8, 4200, 128, 4160, 0, [4190]),   # 64 and 65 tiles a segment
    (15, 2, 1, 130, 64, 100, 1, list(range(0, 130, 9))), (16, 2, 1, 130, 64, 100, 1, list(range(0, 130, 9)) + [130]),
]


def cache(B, S, Hkv, D, lens, window, n_sink, seed, poison=float("nan")):
    """Keys and values whose rows nobody sees are poisoned."""
    g = torch.Generator(DEV).manual_seed(seed)
    k, v = (torch.randn(B, S, Hkv, D, device=DEV, generator=g).bfloat16() for _ in range(2))
    j, n = torch.arange(S, device=DEV)[None], torch.tensor(lens, device=DEV)[:, None]
    hidden = ~((j < n) & ((j > n - 1 - window) | (j < n_sink)))
    for t in (k, v):
        t[hidden] = poison
    return k, v, torch.tensor(lens, dtype=torch.int32, device=DEV)


def check_decode(O, lse, q, k, v, lens, window, n_sink):
    Or, lr, size = sink.decode(np64(q), np64(k), np64(v), lens, window, n_sink)
    close(O, Or, (U + F) * size + U * np.abs(Or), "O")
    empty = np.asarray(lens) == 0
    assert (np64(lse)[empty] == -np.inf).all()
    close(lse[~torch.from_numpy(empty)], lr[~empty], 2 * F, "lse")


@pytest.mark.parametrize("case", DECODE, ids=lambda c: "B{}H{}kv{}S{}D{}w{}s{}".format(*c))
@pytest.mark.parametrize("poison", [float("nan"), float("inf")])
def test_decode(case, poison):
    B, H, Hkv, S, D, window, n_sink, lens = case
    k, v, n = cache(B, S, Hkv, D, lens, window, n_sink, 71, poison)
    q = torch.randn(B, H, D, device=DEV, generator=torch.Generator(DEV).manual_seed(72)).bfloat16()
    ws = torch.full((dfa.dfa_attn_decode_sink_workspace_size(B, H, Hkv, D),), 0xFF, dtype=torch.uint8, device=DEV)
    O, lse = dfa.dfa_attn_decode_sink(q, k, v, n, window, n_sink, workspace_buf=ws)
    dfa.dfa_check_errors()
    check_decode(O, lse, q, k, v, lens, window, n_sink)
    O2, lse2 = dfa.dfa_attn_decode_sink(q, k, v, n, window, n_sink)
    assert torch.equal(O, O2) and torch.equal(lse, lse2)


def test_decode_strided_cache_and_lengths_out_of_range():
    B, H, Hkv, S, D = 3, 4, 2, 200, 128
    g = torch.Generator(DEV).manual_seed(73)
    both = torch.randn(B, Hkv, S, 2, D + 8, device=DEV, generator=g).bfloat16()     # head-major, k and v interleaved
    k, v = both[..., 0, :D].transpose(1, 2), both[..., 1, :D].transpose(1, 2)
    q = torch.randn(B, H, D, device=DEV, generator=g).bfloat16()
    n = torch.tensor([-4, 150, 999], dtype=torch.int32, device=DEV)
    O, lse = dfa.dfa_attn_decode_sink(q, k, v, n, 60, 3)
    dfa.dfa_check_errors()
    check_decode(O, lse, q, k, v, [0, 150, 200], 60, 3)


def test_decode_strides_of_dimensions_of_one_element():
    """They are never used and may be 0; a cache that a batch shares by a stride of 0 is refused."""
    S, D = 150, 64
    k, v, n = cache(1, S, 1, D, [140], 60, 3, 76)
    q = torch.randn(1, 4, D, device=DEV, generator=torch.Generator(DEV).manual_seed(77)).bfloat16()
    flat = [t[0, :, 0].as_strided((1, S, 1, D), (0, D, 0, 1)) for t in (k, v)]
    O, lse = dfa.dfa_attn_decode_sink(q, *flat, n, 60, 3)
    dfa.dfa_check_errors()
    check_decode(O, lse, q, k, v, [140], 60, 3)
    with pytest.raises(dfa.DfaError, match="broadcast"):
        dfa.dfa_attn_decode_sink(q.expand(2, 4, D).contiguous(), k.expand(2, S, 1, D), v.expand(2, S, 1, D), n.repeat(2), 60, 3)


def test_decode_follows_the_prompt_and_is_captured_once():
    """A prompt through the forward, then tokens one at a time through one
    captured call: each row is what the forward gives for the whole sequence."""
    B, H, Hkv, D, W, N, P, T = 2, 8, 2, 128, 100, 4, 180, 260
    q, k, v, _ = make(B, H, Hkv, T, D, torch.bfloat16, device=DEV, seed=74)
    O, lse = dfa.dfa_attn_fwd_sink(q, k, v, W, N)
    kc, vc = torch.full((2, B, 300, Hkv, D), float("nan"), dtype=torch.bfloat16, device=DEV)
    kc[:, :P], vc[:, :P] = k[:, :P], v[:, :P]
    qt = torch.empty(B, H, D, dtype=torch.bfloat16, device=DEV)
    n = torch.full((B,), P, dtype=torch.int32, device=DEV)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, ls = dfa.dfa_attn_decode_sink(qt, kc, vc, n, W, N)
    for i in range(P, T):
        kc[:, i], vc[:, i], qt[:] = k[:, i], v[:, i], q[:, i]
        n.fill_(i + 1)
        graph.replay()
        # both sides round P and the result; the terms' magnitudes are below 4 here
        assert (out.float() - O[:, i].float()).abs().max() <= 4 * U * 4
        assert (ls - lse[:, :, i]).abs().max() <= 4 * F
    dfa.dfa_check_errors()


def test_decode_on_two_streams():
    sets = []
    for z, case in enumerate(DECODE[4:8]):
        B, H, Hkv, S, D, window, n_sink, lens = case
        k, v, n = cache(B, S, Hkv, D, lens, window, n_sink, 80 + z)
        q = torch.randn(B, H, D, device=DEV, generator=torch.Generator(DEV).manual_seed(z)).bfloat16()
        sets.append((q, k, v, n, window, n_sink))
    want = [dfa.dfa_attn_decode_sink(*s) for s in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    for _ in range(10):
        got = [dfa.dfa_attn_decode_sink(*s, stream=st) for s, st in zip(sets, streams)]
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_decode_cache_beyond_32_bits():
    B, H, Hkv, S, D, W, N = 3, 16, 8, 1 << 20, 128, 700, 4
    g = torch.Generator(DEV).manual_seed(75)
    k = torch.empty(B, S, Hkv, D, dtype=torch.bfloat16, device=DEV).normal_(generator=g)
    v = torch.empty(B, S, Hkv, D, dtype=torch.bfloat16, device=DEV).normal_(generator=g)
    q = torch.randn(B, H, D, device=DEV, generator=g).bfloat16()
    lens = [S, 5, S - 1]
    O, lse = dfa.dfa_attn_decode_sink(q, k, v, torch.tensor(lens, dtype=torch.int32, device=DEV), W, N)
    dfa.dfa_check_errors()
    for b, n in enumerate(lens):
        idx = torch.arange(n, device=DEV)
        idx = idx[(idx > n - 1 - W) | (idx < N)]
        # the visible rows alone, all of them in the window
        check_decode(O[b:b + 1], lse[b:b + 1], q[b:b + 1], k[b:b + 1, idx], v[b:b + 1, idx], [idx.numel()], idx.numel(), 0)


# ------------------------------------------------------------------------------------------------ streams, graphs
def step(q, k, v, do, W, N, stream=None):
    Hkv = k.shape[2]
    O, lse = dfa.dfa_attn_fwd_sink(q, k, v, W, N, stream=stream)
    g = dfa.dfa_attn_bwd_sink(q, k, v, O, lse, do, W, N, stream=stream)
    ckpt = dfa.dfa_ckpt8_save(q, k, v, O, stream=stream)
    h = dfa.dfa_attn_bwd_ckpt8(ckpt, lse, do, Hkv, W, N, stream=stream)
    return (O, lse) + g + h


def same_step(a, b):
    for z, (x, y) in enumerate(zip(a, b)):
        if z in (2, 5):      # dQ: fp32 atomics
            torch.testing.assert_close(x.float(), y.float(), rtol=2 * U, atol=2e-3)
        else:
            assert torch.equal(x, y), z


def test_captured_and_replayed():
    W, N = 200, 4
    q, k, v, do = make(1, 4, 2, 1300, 128, torch.bfloat16, device=DEV, seed=51)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):        # captured without an eager call before it
        out = step(q, k, v, do, W, N)
    for seed in (52, 53):
        for t, n in zip((q, k, v, do), make(1, 4, 2, 1300, 128, torch.bfloat16, device=DEV, seed=seed)):
            t.copy_(n)
        g.replay()
        torch.cuda.synchronize()
        same_step(out, step(q, k, v, do, W, N))
    dfa.dfa_check_errors()


def test_captured_on_a_stream_of_its_own():
    """A stream that a captured one forks: what the calls allocate there belongs to the graph."""
    W, N = 90, 2
    sets = [make(1, 4, 2, 700, D, torch.bfloat16, device=DEV, seed=91) for D in (64, 128)]
    g, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.graph(g):
        now = torch.cuda.current_stream()
        side.wait_stream(now)
        out = [step(*sets[0], W, N), step(*sets[1], W, N, stream=side)]
        kept = dfa.dfa_attn_fwd_sink(*sets[1][:3], W, N, stream=side)[0]      # the other output is dropped in the capture
        now.wait_stream(side)
    for seed in (92, 93):
        for tensors, D in zip(sets, (64, 128)):
            for t, n in zip(tensors, make(1, 4, 2, 700, D, torch.bfloat16, device=DEV, seed=seed)):
                t.copy_(n)
        g.replay()
        torch.cuda.synchronize()
        for got, tensors in zip(out, sets):
            same_step(got, step(*tensors, W, N))
        assert torch.equal(kept, out[1][0])
    dfa.dfa_check_errors()


FIRST = """
import torch
from long_context_causal_gb300 import dfa
from long_context_causal_gb300.inputs import make
q, k, v, do = make(1, 1, 1, 2000, 64, torch.bfloat16, device="cuda", seed=90)
lens = torch.full((1,), 1999, dtype=torch.int32, device="cuda")
q1 = q[:, 1998].contiguous()

def chain():
    O, lse = dfa.dfa_attn_fwd_sink(q, k, v, 2000)             # blocks shared by clusters
    O2, lse2 = dfa.dfa_attn_fwd_sink(q, k, v, 40, 3)
    kept = dfa.dfa_ckpt8_save(q, k, v, O2)
    return (O, lse, O2, lse2, kept) + dfa.dfa_attn_bwd_ckpt8(kept, lse2, do, 1, 40, 3)[1:] + \\
        dfa.dfa_attn_decode_sink(q1, k, v, lens, 40, 3)

torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    got = chain()
graph.replay()
torch.cuda.synchronize()
assert all(torch.equal(a, b) for a, b in zip(got, chain()))
dfa.dfa_check_errors()
"""


def test_first_calls_inside_a_capture():
    """What a kernel sets up once per device may be set up while a stream is captured."""
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", FIRST], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]


def test_another_stream_and_two_at_once():
    W, N = 150, 3
    sets = [make(1, 4, 2, 1100, D, torch.bfloat16, device=DEV, seed=54 + D) for D in (64, 128)]
    want = [step(*s, W, N) for s in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    for _ in range(5):
        got = [step(*s, W, N, stream=st) for s, st in zip(sets, streams)]
        for st in streams:
            st.synchronize()
        for a, b in zip(got, want):
            same_step(a, b)
    got = step(*sets[0], W, N, stream=streams[0].cuda_stream)     # a raw handle
    streams[0].synchronize()
    same_step(got, want[0])


DELAY = 40_000_000      # cycles, about 20 ms: longer than what the host does meanwhile


def test_memory_of_calls_on_another_stream():
    """A call on another stream may not write memory that the current one has still to write, nor read or leave
    memory that the current one takes again when the caller drops a tensor."""
    W, N, Hkv = 150, 3, 2
    q, k, v, do = make(1, 4, Hkv, 1100, 64, torch.bfloat16, device=DEV, seed=59)
    lens, q1 = torch.full((1,), 900, dtype=torch.int32, device=DEV), q[:, 899].contiguous()

    def chain(stream=None):
        out = step(q, k, v, do, W, N, stream=stream)
        ckpt = dfa.dfa_ckpt8_save(q, k, v, out[0], stream=stream)
        return out + dfa.dfa_ckpt8_restore(ckpt, 1, 4, Hkv, 1100, 64, stream=stream) + \
            dfa.dfa_attn_decode_sink(q1, k, v, lens, W, N, stream=stream)

    want, now, s = chain(), torch.cuda.current_stream(), torch.cuda.Stream()
    other = q.flip(1).contiguous()
    for _ in range(3):
        # outputs: blocks of their sizes that the current stream is about to fill
        torch.cuda.synchronize()
        blocks = [torch.empty_like(t) for t in want]
        torch.cuda._sleep(DELAY)
        for t in blocks:
            t.fill_(7)
        del blocks
        got = chain(s)
        torch.cuda.synchronize()
        same_step(got[:8], want[:8])
        assert all(torch.equal(a, b) for a, b in zip(got[8:], want[8:]))
        # inputs that are dropped while the other stream has still to read them
        ckpt = dfa.dfa_ckpt8_save(q, k, v, want[0])
        rest = [t.clone() for t in (want[1], do)]
        s.wait_stream(now)
        with torch.cuda.stream(s):
            torch.cuda._sleep(DELAY)
        got = dfa.dfa_attn_bwd_ckpt8(ckpt, *rest, Hkv, W, N, stream=s)
        sizes = [torch.empty_like(t, device="meta") for t in (ckpt, *rest)]
        del ckpt, rest
        blocks = [torch.full_like(t, 1, device=DEV) for t in sizes]
        torch.cuda.synchronize()
        assert torch.equal(got[1], want[6]) and torch.equal(got[2], want[7])
        # an output that is dropped while the current stream has still to read it
        O, lse = dfa.dfa_attn_fwd_sink(q, k, v, W, N, stream=s)
        s.synchronize()
        torch.cuda._sleep(DELAY)
        seen = O.clone()
        del O, lse
        dfa.dfa_attn_fwd_sink(other, k, v, W, N, stream=s)
        torch.cuda.synchronize()
        assert torch.equal(seen, want[0])
    dfa.dfa_check_errors()


def test_tensors_on_the_wrong_place_are_refused():
    q, k, v, do = make(1, 2, 1, 64, 64, torch.bfloat16, device=DEV, seed=57)
    with pytest.raises(ValueError, match="CUDA"):
        dfa.dfa_attn_fwd_sink(q, k.cpu(), v, 4)
    with pytest.raises(dfa.DfaError):
        dfa.dfa_attn_fwd_sink(q.float(), k.float(), v.float(), 4)
    with pytest.raises(ValueError, match="O must be"):
        dfa.dfa_attn_fwd_sink(q, k, v, 4, O=torch.empty(1, 63, 2, 64, dtype=torch.bfloat16, device=DEV))
    with pytest.raises(ValueError, match="workspace"):
        dfa.dfa_attn_bwd_sink(q, k, v, q, torch.zeros(1, 2, 64, device=DEV), do, 4, workspace_buf=torch.zeros(9, device=DEV))
    empty = dfa.dfa_attn_fwd_sink(q[:, :0], k[:, :0], v[:, :0], 4)
    assert empty[0].shape == (1, 0, 2, 64) and empty[1].shape == (1, 2, 0)


@pytest.mark.parametrize("n_sink", [0, 4])
@pytest.mark.parametrize("B,S", [(0, 300), (2, 0)])
def test_empty_batches(B, S, n_sink):
    H, Hkv, D, W = 4, 2, 64, 100
    q, do = (torch.empty(B, S, H, D, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    k, v = (torch.empty(B, S, Hkv, D, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    O, lse = dfa.dfa_attn_fwd_sink(q, k, v, W, n_sink)
    ckpt = dfa.dfa_ckpt8_save(q, k, v, O)
    for grads in (dfa.dfa_attn_bwd_sink(q, k, v, O, lse, do, W, n_sink), dfa.dfa_attn_bwd_ckpt8(ckpt, lse, do, Hkv, W, n_sink)):
        assert [t.shape for t in grads] == [q.shape, k.shape, k.shape]
    assert [t.shape for t in dfa.dfa_ckpt8_restore(ckpt, B, H, Hkv, S, D)] == [q.shape, k.shape, k.shape, q.shape]
    if B == 0:
        n = torch.empty(0, dtype=torch.int32, device=DEV)
        O, lse = dfa.dfa_attn_decode_sink(torch.empty(0, H, D, dtype=torch.bfloat16, device=DEV), k, v, n, W, n_sink)
        assert O.shape == (0, H, D) and lse.shape == (0, H)
    dfa.dfa_check_errors()


def test_numbers_out_of_range_are_refused():
    q, k, v, do = make(1, 2, 1, 64, 64, torch.bfloat16, device=DEV, seed=58)
    lens = torch.full((1,), 64, dtype=torch.int32, device=DEV)
    for bad in (1 << 31, -(1 << 31) - 1, 1 << 40):
        with pytest.raises(ValueError, match="32-bit"):
            dfa.dfa_attn_fwd_sink(q, k, v, bad)
        with pytest.raises(ValueError, match="32-bit"):
            dfa.dfa_attn_decode_sink(q[:, 0].contiguous(), k, v, lens, 4, bad)
    with pytest.raises(OverflowError):
        dfa.dfa_attn_fwd_sink(q, k, v, 1 << 70)
    for bad in (1.5, None, "4"):
        with pytest.raises(TypeError):
            dfa.dfa_attn_fwd_sink(q, k, v, bad)
    for window, n_sink in ((0, 0), (-3, 0), (4, -1), (4, 129)):
        with pytest.raises(dfa.DfaError):
            dfa.dfa_attn_fwd_sink(q, k, v, window, n_sink)
    for scale in (0.0, -1.0, float("nan"), 1e300):
        with pytest.raises(dfa.DfaError):
            dfa.dfa_attn_fwd_sink(q, k, v, 4, scale=scale)
    with pytest.raises(TypeError):
        dfa.dfa_attn_fwd_sink(q, k, [1, 2], 4)
    with pytest.raises(AttributeError):
        dfa.dfa_attn_fwd_sink(q, k, v, 4, stream="none")


def test_calls_from_several_threads():
    """Each thread on a stream of its own; the calls let other threads run."""
    import threading
    cases = [(1, 4, 2, 700, 64, 100, 4), (1, 2, 2, 1500, 128, 1500, 0), (2, 8, 2, 300, 128, 40, 1), (1, 1, 1, 2500, 64, 900, 17)]
    data = [make(*c[:5], torch.bfloat16, device=DEV, seed=80 + i) for i, c in enumerate(cases)]
    want = [step(*d, *c[5:]) for d, c in zip(data, cases)]
    torch.cuda.synchronize()
    failed = []

    def work(i):
        try:
            s = torch.cuda.Stream()
            with torch.cuda.stream(s):
                for _ in range(20):
                    same_step(step(*data[i], *cases[i][5:]), want[i])
        except BaseException as e:       # shown by the test, not lost with the thread
            failed.append((cases[i], e))

    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(cases))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    dfa.dfa_check_errors()
    assert not failed, failed


def test_offsets_beyond_32_bits():
    """512K tokens of 32 heads: 2^31 elements in q, and dQ's fp32 accumulator.
    Rows of the last head and sequence end against the reference on the slice
    that they see."""
    B, H, Hkv, S, D, W, N = 1, 32, 8, 524288 + 77, 128, 300, 4
    g = torch.Generator(DEV).manual_seed(61)
    q, k, v, do = (torch.empty(B, S, h, D, dtype=torch.bfloat16, device=DEV).normal_(generator=g) for h in (H, Hkv, Hkv, H))
    O, lse = dfa.dfa_attn_fwd_sink(q, k, v, W, N)
    dQ, dK, dV = dfa.dfa_attn_bwd_sink(q, k, v, O, lse, do, W, N)
    ckpt = dfa.dfa_ckpt8_save(q, k, v, O)
    back = dfa.dfa_ckpt8_restore(ckpt, B, H, Hkv, S, D)
    dfa.dfa_check_errors()
    for got, t in zip(back, (q, k, v, O)):
        assert np.array_equal(np64(got[:, -200:, -1]), sink.ckpt8(np64(t[:, -200:, -1])))
    G = H // Hkv
    a = S - 1000                          # keys [a, S) and the sinks, queries from a + W - 1 on see no other
    idx = torch.cat((torch.arange(N, device=DEV), torch.arange(a, S, device=DEV)))
    hs, gs = slice(H - G, H), slice(Hkv - 1, Hkv)
    sub = [np64(t[:, idx][:, :, s]) for t, s in ((q, hs), (k, gs), (v, gs), (O, hs))]
    sd, sl = np64(do[:, idx][:, :, hs]), np64(lse[:, hs][:, :, idx])
    # in the slice the keys of the sinks come first and the window is the same
    Or, lr, size = sink.attn_fwd(*sub[:3], W, N)
    rows = slice(N + W - 1, None)
    close(O[:, a + W - 1:, hs], Or[:, rows], ((U + F) * size + U * np.abs(Or))[:, rows], "O")
    close(lse[:, hs, a + W - 1:], lr[:, :, rows], 2 * F, "lse")
    ref = sink.attn_bwd(*sub, sl, sd, W, N)
    for got, name in ((dQ[:, a + W - 1:, hs], "dQ"), (dK[:, a + W - 1:, gs], "dK"), (dV[:, a + W - 1:, gs], "dV")):
        r, terms, cancel, floor = (t[:, rows] for t in ref[name])
        close(got, r, ((1 if name == "dV" else 2) * U + F) * terms + F2 * cancel + 2.0 ** -39 * floor + U * np.abs(r) + 1e-30, name)
