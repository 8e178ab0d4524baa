"""The calls over a long cache on the GPU, against the fp64 reference (oracle/cache.py).

Tolerances count what is rounded.  fp32 sums of up to D = 128 products move a score
by less than F / 2 = 2^-13 (scores here stay below 60), a log-sum-exp by as much; a
weight exp(s - lse) by F times itself where lse is handed in, by 2 F where it is the
call's own.  Weights are positive, so sums of them are off by no more, and by 2^-24
per addition (at most 2^10 of these in a row in one sum here: F / 4).  O, as in the
windowed tests: P is rounded to bf16 (U times the sum of P |v|) and the result once.
What is kept, moved and counted is exact.
"""
import numpy as np
import pytest
import torch

from long_context_causal_gb300 import dfa
from oracle import cache, sink

pytestmark = pytest.mark.gpu
DEV = "cuda"
U, F = 2.0 ** -8, 2.0 ** -12
NAN = float("nan")


def np64(t):
    return t.detach().double().cpu().numpy()


def close(got, ref, tol, what):
    bad = ~(np.abs(np64(got) - ref) <= tol)
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size}, first at {np.argwhere(bad)[0]}, worst {np.nanmax(np.abs(np64(got) - ref) / (tol + 1e-30)):.3g} of the tolerance"


def gen(seed):
    return torch.Generator(DEV).manual_seed(seed)


def rand(seed, *shape, dtype=torch.bfloat16):
    return torch.randn(*shape, device=DEV, generator=gen(seed)).to(dtype)


def lens_of(lens):
    return torch.tensor(lens, dtype=torch.int32, device=DEV)


# ------------------------------------------------------------------------------------------------ masses of a prompt
# (B, H, Hkv, S, D, window, n_sink, n_last)
MASS = [
    (1, 1, 1, 1, 64, 1, 0, 1), (2, 2, 1, 2, 128, 1, 1, 2), (1, 4, 2, 31, 64, 31, 0, 7), (2, 4, 4, 127, 128, 127, 0, 127),
    (1, 6, 2, 128, 64, 16, 4, 128), (3, 3, 3, 129, 128, 129, 0, 1), (2, 8, 2, 300, 64, 300, 0, 300), (1, 8, 1, 513, 128, 100, 128, 513),
    (1, 4, 2, 700, 64, 1, 3, 700), (1, 2, 2, 1025, 128, 1025, 0, 64), (2, 6, 2, 1100, 64, 512, 17, 1099), (1, 5, 5, 1500, 128, 1500, 0, 1500),
    (1, 8, 2, 2000, 64, 130, 1, 333), (1, 3, 1, 2500, 128, 700, 4, 2500), (1, 2, 1, 2600, 64, 2000, 0, 129), (1, 4, 2, 2048, 128, 128, 128, 2048),
    (1, 1, 1, 4200, 64, 40, 9, 4200), (2, 4, 1, 900, 128, 900, 0, 128), (1, 8, 1, 1300, 64, 300, 5, 64), (3, 2, 2, 640, 128, 100, 128, 512),
    (1, 3, 1, 1000, 64, 1000, 0, 65), (2, 16, 1, 2100, 128, 64, 3, 1), (1, 12, 4, 3001, 64, 2000, 0, 33), (5, 4, 4, 130, 128, 130, 0, 2),
]
MASS_IDS = ["B{}H{}kv{}S{}D{}w{}s{}l{}".format(*c) for c in MASS]


def prompt(case, seed):
    B, H, Hkv, S, D, window, n_sink, n_last = case
    q, k = rand(seed, B, S, H, D), rand(seed + 1, B, S, Hkv, D)
    k[:, ::7] *= 2
    lse = torch.from_numpy(sink.attn_fwd(np64(q), np64(k), np64(k), window, n_sink)[1]).float().to(DEV)
    return q, k, lse


def poison(case, q, k, lse):
    """NaN in what no counted query needs: earlier queries and their lse, and the keys that none of the others sees."""
    B, H, Hkv, S, D, window, n_sink, n_last = case
    q, k, lse = q.clone(), k.clone(), lse.clone()
    q[:, :S - n_last], lse[:, :, :S - n_last] = NAN, NAN
    k[:, torch.from_numpy(~sink.visible(S, window, n_sink)[S - n_last:].any(0)).to(DEV)] = NAN
    return q, k, lse


@pytest.mark.parametrize("case", MASS, ids=MASS_IDS)
def test_mass(case):
    window, n_sink, n_last = case[5:]
    q, k, lse = prompt(case, 51)
    ref = cache.mass(np64(q), np64(k), np64(lse), window, n_sink, n_last)
    bad = poison(case, q, k, lse)
    ws = torch.full((dfa.dfa_attn_mass_workspace_size(*case[:5]),), 0xFF, dtype=torch.uint8, device=DEV)
    got = dfa.dfa_attn_mass(*bad, window, n_sink, n_last, workspace_buf=ws)
    dfa.dfa_check_errors()
    # a score is a sum of D products, its weight off by F / 2 relative; the sums by a quarter of F
    close(got, ref, F * ref, "mass")
    assert torch.equal(got, dfa.dfa_attn_mass(q, k, lse, window, n_sink, n_last))


def test_mass_what_it_must_not_trip_over():
    """A row that sees nothing (lse = -inf) counts for nothing; a NaN query reaches the keys that it sees and no others;
    weights far above and below one; a scale of the caller's."""
    case = (1, 2, 1, 900, 64, 200, 3, 900)
    q, k, lse = prompt(case, 53)
    lse[0, 1, 700] = -float("inf")
    got = dfa.dfa_attn_mass(q, k, lse, 200, 3)
    ref = cache.mass(np64(q), np64(k), np.where(np64(lse) == -np.inf, np.inf, np64(lse)), 200, 3, 900)
    close(got, ref, F * ref, "mass")
    q[0, 500, 0] = NAN
    with_nan, seen = dfa.dfa_attn_mass(q, k, lse, 200, 3)[0, 0], torch.from_numpy(sink.visible(900, 200, 3)[500]).to(DEV)
    assert with_nan[seen].isnan().all() and torch.equal(with_nan[~seen], got[0, 0][~seen])
    q, k, lse = prompt(case, 54)
    got = dfa.dfa_attn_mass(q, k, lse - 40, 200, 3, scale=0.5)
    ref = cache.mass(np64(q), np64(k), np64(lse) - 40, 200, 3, 900, 0.5)
    close(got, ref, F * ref, "mass")


# (B, H, Hkv, S, D, window, n_sink, n_last): by a cluster per block, by all SMs, by the kernels of few queries (their
# groups of 128 columns: 1, 2, 4)
@pytest.mark.parametrize("case", [(1, 2, 1, 900, 64, 200, 3, 900), (2, 8, 2, 6000, 128, 1500, 5, 6000), (1, 2, 2, 5000, 64, 5000, 0, 3000),
                                  (1, 2, 1, 900, 128, 200, 3, 50), (2, 4, 1, 1500, 64, 300, 0, 64), (1, 8, 2, 700, 128, 700, 0, 100)],
                         ids=lambda c: "B{}H{}kv{}S{}D{}w{}s{}l{}".format(*c))
def test_mass_of_a_nan_query_reaches_the_keys_it_sees(case):
    """With the log-sum-exp that the windowed forward gives for it; one lower than 32 bits times log2 e hold likewise."""
    B, H, Hkv, S, D, window, n_sink, n_last = case
    q, k = rand(57, B, S, H, D), rand(58, B, S, Hkv, D)
    _, lse = dfa.dfa_attn_fwd_sink(q, k, k, window, n_sink)
    want = dfa.dfa_attn_mass(q, k, lse, window, n_sink, n_last)
    for i in (S - 1, S - n_last // 2, S - n_last):
        bad = q.clone()
        bad[0, i, 0, 5] = NAN
        _, lse_bad = dfa.dfa_attn_fwd_sink(bad, k, k, window, n_sink)
        assert lse_bad[0, 0, i].isnan() and lse_bad.isnan().sum() == 1
        low = lse.clone()
        low[0, 0, i] = -3.4e38
        seen = torch.zeros(B, Hkv, S, dtype=torch.bool, device=DEV)
        seen[0, 0] = torch.arange(S, device=DEV) <= i
        seen[0, 0, n_sink:max(i - window + 1, n_sink)] = False
        for got, there in ((dfa.dfa_attn_mass(bad, k, lse_bad, window, n_sink, n_last), torch.isnan),
                           (dfa.dfa_attn_mass(q, k, lse_bad, window, n_sink, n_last), torch.isnan),
                           (dfa.dfa_attn_mass(q, k, low, window, n_sink, n_last), torch.isposinf)):
            assert torch.equal(there(got), seen), i
            assert torch.equal(got[~seen], want[~seen])
    dfa.dfa_check_errors()


@pytest.mark.parametrize("case", [(1, 2, 1, 900, 64, 200, 3, 900), (2, 8, 2, 6001, 128, 1500, 5, 6001), (1, 2, 1, 900, 128, 200, 3, 50),
                                  (2, 4, 1, 1507, 64, 300, 0, 61), (1, 8, 2, 700, 128, 700, 0, 100), (1, 16, 1, 1300, 128, 1300, 0, 20)],
                         ids=lambda c: "B{}H{}kv{}S{}D{}w{}s{}l{}".format(*c))
def test_mass_of_keys_whose_scores_are_below_32_bits(case):
    """Keys with an infinity and a score of -inf draw nothing.  Tiles of queries that end behind the sequence have rows of
    zeros there, whose products with such a key are NaN."""
    B, H, Hkv, S, D, window, n_sink, n_last = case
    q, k, lse = rand(59, B, S, H, D), rand(60, B, S, Hkv, D), rand(61, B, H, S, dtype=torch.float32) + 8
    q[..., 3] = q[..., 3].abs() + 1
    want = dfa.dfa_attn_mass(q, k, lse, window, n_sink, n_last)
    far = torch.zeros(S, dtype=torch.bool, device=DEV)
    far[[0, S // 2, S - 300, S - 130, S - 3, S - 1]] = True
    k[:, far, :, 3] = -float("inf")
    got = dfa.dfa_attn_mass(q, k, lse, window, n_sink, n_last)
    dfa.dfa_check_errors()
    assert (got[..., far] == 0).all() and torch.equal(got[..., ~far], want[..., ~far])


def test_mass_of_many_heads_and_blocks():
    """More blocks than SMs, most of them swept whole, and a few that many CTAs share: every query gives away one."""
    from long_context_causal_gb300.inputs import make
    for B, H, Hkv, S, D, window, n_sink in ((2, 8, 4, 30000, 64, 700, 5), (1, 4, 2, 20001, 128, 20001, 0), (70, 4, 4, 515, 64, 515, 0)):
        q, k, v, _ = make(B, H, Hkv, S, D, torch.bfloat16, device=DEV, seed=55)
        O, lse = dfa.dfa_attn_fwd_sink(q, k, v, window, n_sink)
        for n_last in (S, 1000 if S > 1000 else 1):
            got = dfa.dfa_attn_mass(q, k, lse, window, n_sink, n_last)
            dfa.dfa_check_errors()
            np.testing.assert_allclose(np64(got).sum((1, 2)), H * n_last, rtol=4 * F)
            # keys of every block against the definition, all queries that see them
            for j in list(range(0, S, S // 9 + 1)) + [0, S - 1]:
                lo = max(j, S - n_last)
                i = torch.arange(lo, max(lo, S if j < n_sink else min(j + window, S)), device=DEV)
                s = torch.einsum("bihd,bhd->bhi", q[:, i].double(), k[:, j].double().repeat_interleave(H // Hkv, 1)) * D ** -0.5
                w = torch.exp(s - lse[:, :, i].double()).sum(2).reshape(B, Hkv, -1).sum(2)
                close(got[:, :, j], np64(w), 2 * F * np64(w), "mass")


# ------------------------------------------------------------------------------------------------ single tokens with masses
# (B, H, Hkv, S, D, window, n_sink, lens)
STEP = [
    (1, 1, 1, 1, 64, 1, 0, [1]), (2, 2, 1, 3, 128, 3, 0, [0, 2]), (1, 8, 2, 64, 128, 64, 0, [64]),
    (2, 8, 8, 65, 64, 65, 0, [65, 64]), (3, 12, 4, 200, 128, 60, 3, [200, 61, 62]), (2, 16, 1, 300, 64, 100, 128, [300, 129]),
    (1, 17, 1, 130, 128, 130, 0, [127]), (2, 40, 2, 500, 64, 77, 17, [500, 90]), (2, 33, 3, 257, 128, 16, 1, [257, 1]),
    (1, 4, 4, 5000, 128, 5000, 0, [4999]), (1, 32, 8, 9000, 64, 9000, 0, [8577]), (6, 8, 2, 3001, 128, 1500, 4, [0, 1, 1500, 1501, 3001, 2222]),
    (40, 8, 4, 700, 64, 700, 0, [i * 17 for i in range(40)]),
]


def poisoned(case, seed):
    B, H, Hkv, S, D, window, n_sink, lens = case
    q, k, v, m = rand(seed, B, H, D), rand(seed + 1, B, S, Hkv, D), rand(seed + 2, B, S, Hkv, D), rand(seed + 3, B, Hkv, S, dtype=torch.float32).abs()
    k[:, ::7] *= 2
    for b, n in enumerate(lens):       # what the query does not see may hold anything
        j = torch.arange(S, device=DEV)
        hidden = (j >= n) | ((j <= n - 1 - window) & (j >= n_sink))
        k[b, hidden], v[b, hidden] = NAN, float("inf")
        m[b, :, n:] = NAN
    return q, k, v, lens_of(lens), m


def check_step(got, case, q, k, v, m):
    B, H, Hkv, S, D, window, n_sink, lens = case
    O, lse, out = got
    Or, lr, size = sink.decode(np64(q), np64(k), np64(v), lens, window, n_sink)
    close(O, Or, (U + F) * size + U * np.abs(Or), "O")
    empty = np.asarray(lens) == 0
    assert (np64(lse)[empty] == -np.inf).all()
    close(lse[~torch.from_numpy(empty)], lr[~empty], 2 * F, "lse")
    w = cache.step_mass(np64(q), np64(k), lens, window, n_sink)
    live = np.arange(S) < np.asarray(lens)[:, None, None]
    before = np.zeros_like(w) if m is None else np.where(live, np64(m), 0.0)
    close(out, before + w, 2 * F * w + 2.0 ** -23 * (before + w), "mass")
    assert (np64(out)[~np.broadcast_to(live, w.shape)] == 0).all()


@pytest.mark.parametrize("case", STEP, ids=lambda c: "B{}H{}kv{}S{}D{}w{}s{}".format(*c))
def test_step_masses(case):
    q, k, v, n, m = poisoned(case, 11)
    window, n_sink = case[5:7]
    got = dfa.dfa_attn_decode_mass(q, k, v, n, m, window, n_sink)
    alone = dfa.dfa_attn_decode_mass(q, k, v, n, None, window, n_sink)
    dfa.dfa_check_errors()
    check_step(got, case, q, k, v, m)
    check_step(alone, case, q, k, v, None)
    # the same bits in place and again
    into = m.clone()
    again = dfa.dfa_attn_decode_mass(q, k, v, n, into, window, n_sink, mass_out=into)
    assert again[2] is into or again[2].data_ptr() == into.data_ptr()
    for a, b, c in zip(got[:2], again[:2], alone[:2]):
        assert torch.equal(a, b) and torch.equal(a, c)
    assert torch.equal(again[2], got[2])


def test_step_masses_strided_cache_and_lengths_out_of_range():
    B, H, Hkv, S, D = 3, 4, 2, 200, 128
    both = rand(21, B, Hkv, S, 2, D + 8)           # head-major, k and v interleaved
    k, v = both[..., 0, :D].transpose(1, 2), both[..., 1, :D].transpose(1, 2)
    q, m = rand(22, B, H, D), rand(23, B, Hkv, S, dtype=torch.float32)
    got = dfa.dfa_attn_decode_mass(q, k, v, lens_of([-4, 150, 999]), m, 60, 3, scale=0.2)
    dfa.dfa_check_errors()
    Or, lr, size = sink.decode(np64(q), np64(k), np64(v), [0, 150, 200], 60, 3, 0.2)
    close(got[0], Or, (U + F) * size + U * np.abs(Or), "O")
    w = cache.step_mass(np64(q), np64(k), [0, 150, 200], 60, 3, 0.2)
    want = np.where(np.arange(S) < np.array([0, 150, 200])[:, None, None], np64(m), 0.0) + w
    close(got[2], want, 2 * F * w + 2.0 ** -23 * np.abs(want), "mass")


def test_step_masses_of_a_cache_beyond_32_bits():
    B, H, Hkv, S, D, W, N = 3, 16, 8, 1 << 20, 128, 700, 4
    k, v = (torch.empty(B, S, Hkv, D, dtype=torch.bfloat16, device=DEV).normal_(generator=gen(24 + i)) for i in range(2))
    q, lens = rand(26, B, H, D), [S, 5, S - 1]
    for window in (W, None):
        got = dfa.dfa_attn_decode_mass(q, k, v, lens_of(lens), None, window, N)
        dfa.dfa_check_errors()
        # every head of a sequence gives away one
        np.testing.assert_allclose(np64(got[2]).sum((1, 2)), H, rtol=4 * F)
        for b, n in enumerate(lens):
            idx = torch.arange(n, device=DEV)
            idx = idx[(idx > n - 1 - W) | (idx < N)] if window else idx[-2000:]
            s = torch.einsum("hd,jhd->hj", q[b].double(), k[b, idx].double().repeat_interleave(2, 1)) * D ** -0.5
            w = torch.exp(s - got[1][b].double()[:, None]).reshape(Hkv, 2, -1).sum(1)
            close(got[2][b][:, idx], np64(w), 2 * F * np64(w), "mass")


def test_step_masses_of_nans_and_scores_below_32_bits():
    """Visible keys whose score is -inf in 32 bits draw nothing, whole tiles of them too; a NaN score reaches all
    that its head's softmax touches and nothing else.  One launch, a cluster and a second one, all SMs."""
    for case in ((1, 4, 2, 700, 64, 700, 0, [700]), (1, 40, 2, 700, 128, 300, 9, [650]), (3, 8, 2, 6000, 128, 6000, 0, [6000, 64, 5000])):
        B, H, Hkv, S, D, window, n_sink, lens = case
        q, k, v, n, m = poisoned(case, 15)
        q[:, :, 0], k[:, :, :, 0] = 2.0 ** 100, 0
        for b in range(B):
            for lo, hi in ((0, 16), (lens[b] - 200, lens[b] - 70), (lens[b] - 3, lens[b] - 1)):
                k[b, max(lo, 0):max(hi, 0), :, 0] = -2.0 ** 100
        got = dfa.dfa_attn_decode_mass(q, k, v, n, m, window, n_sink)
        dfa.dfa_check_errors()
        check_step(got, case, q, k, v, m)
        j, G = lens[0] - 5, H // Hkv
        k[0, j, 1, 3] = NAN
        O, lse, out = dfa.dfa_attn_decode_mass(q, k, v, n, m, window, n_sink)
        dfa.dfa_check_errors()
        seen = torch.arange(S, device=DEV)
        seen = (seen < lens[0]) & ((seen >= lens[0] - window) | (seen < n_sink))
        assert O[0, G:].isnan().all() and lse[0, G:].isnan().all() and out[0, 1, seen].isnan().all()
        for a, b in ((O[0, :G], got[0][0, :G]), (lse[0, :G], got[1][0, :G]), (out[0, 0], got[2][0, 0]), (out[0, 1, ~seen], got[2][0, 1, ~seen]),
                     (O[1:], got[0][1:]), (out[1:], got[2][1:])):
            assert torch.equal(a, b)


# segments of one CTA each, by a cluster, cut by several CTAs, in two blocks of heads
@pytest.mark.parametrize("case", [(90, 8, 4, 60, 64, 60, 0, [1 + i % 60 for i in range(90)]), (1, 4, 2, 700, 128, 200, 3, [640]),
                                  (3, 8, 2, 6000, 128, 6000, 0, [6000, 64, 5000]), (1, 20, 1, 500, 64, 500, 0, [431]),
                                  (40, 34, 2, 400, 128, 300, 5, [10 * i for i in range(40)])], ids=lambda c: "B{}H{}kv{}S{}D{}".format(*c))
def test_step_of_a_head_whose_scores_are_all_below_32_bits(case):
    """It draws nothing: O = 0, lse = -inf and no weight, whoever has its keys; the other heads' results stay."""
    B, H, Hkv, S, D, window, n_sink, lens = case
    q, k, v, n, m = poisoned(case, 16)
    q[:, :, 0], k[..., 0] = 0, -2.0 ** 100
    whole = dfa.dfa_attn_decode_mass(q, k, v, n, m, window, n_sink)
    steps = dfa.dfa_attn_decode_sink(q, k, v, n, window, n_sink)
    check_step(whole, case, q, k, v, m)
    q[:, 1, 0] = 2.0 ** 100
    others = [h for h in range(H) if h != 1]
    for (O, lse), ref in ((dfa.dfa_attn_decode_mass(q, k, v, n, m, window, n_sink)[:2], whole), (dfa.dfa_attn_decode_sink(q, k, v, n, window, n_sink), steps)):
        dfa.dfa_check_errors()
        assert (O[:, 1] == 0).all() and (lse[:, 1] == -np.inf).all()
        assert torch.equal(O[:, others], ref[0][:, others]) and torch.equal(lse[:, others], ref[1][:, others])
    got = dfa.dfa_attn_decode_mass(q, k, v, n, None, window, n_sink)[2]
    q[:, 1, 0], k[..., 0] = 0, 0                       # the weights of the other heads
    w = cache.step_mass(np64(q), np64(k), lens, window, n_sink)
    w[:, :1] -= cache.step_mass(np64(q[:, 1:2]), np64(k[:, :, :1]), lens, window, n_sink)
    close(got, w, 2 * F * w + 1e-15, "mass")           # w is a difference of fp64 numbers of at most 1 per head and key


def test_prefix_of_a_head_whose_scores_are_all_below_32_bits():
    for B, H, Hkv, P, S, D, lens in ((3, 8, 2, 500, 20, 64, [20, 0, 7]), (5, 12, 4, 700, 400, 128, [400, 0, 64, 7, 399]), (2, 4, 2, 0, 30, 64, [30, 1])):
        q, kp, vp, k, v = rand(96, B, H, D), rand(97, P, Hkv, D), rand(98, P, Hkv, D), rand(99, B, S, Hkv, D), rand(100, B, S, Hkv, D)
        q[:, :, 0], kp[:, :, 0], k[..., 0] = 0, -2.0 ** 100, -2.0 ** 100
        want = dfa.dfa_attn_decode_prefix(q, kp, vp, k, v, lens_of(lens))
        check_prefix(want, q, kp, vp, k, v, lens)
        q[:, 1, 0] = 2.0 ** 100
        O, lse = dfa.dfa_attn_decode_prefix(q, kp, vp, k, v, lens_of(lens))
        dfa.dfa_check_errors()
        assert (O[:, 1] == 0).all() and (lse[:, 1] == -np.inf).all()
        others = [h for h in range(H) if h != 1]
        assert torch.equal(O[:, others], want[0][:, others]) and torch.equal(lse[:, others], want[1][:, others])


# ------------------------------------------------------------------------------------------------ a shared prefix
# (B, H, Hkv, P, S, D, lens): one query tile of a head, two, three, many; few keys and many pieces; own rows from none on
PREFIX = [
    (1, 1, 1, 1, 1, 64, [0]), (2, 2, 1, 0, 3, 128, [0, 2]), (1, 4, 2, 5, 4, 128, [4]), (3, 12, 4, 127, 70, 64, [0, 1, 70]),
    (4, 8, 8, 128, 64, 128, [64, 3, 0, 63]), (2, 34, 2, 300, 65, 64, [65, 0]), (4, 32, 8, 1000, 64, 128, [1, 17, 34, 50]),
    (33, 4, 1, 129, 40, 128, [i for i in range(33)]), (64, 8, 2, 700, 33, 64, [33 - i % 34 for i in range(64)]),
    (97, 4, 1, 1500, 20, 128, [i % 21 for i in range(97)]), (130, 6, 2, 257, 9, 64, [i % 10 for i in range(130)]),
    (7, 40, 1, 4000, 600, 64, [600, 0, 599, 64, 65, 1, 300]), (2, 2, 1, 30000, 129, 128, [129, 0]), (200, 16, 4, 130, 5, 64, [i % 6 for i in range(200)]),
]


def check_prefix(got, q, kp, vp, k, v, lens, scale=None):
    Or, lr, size = cache.decode_prefix(np64(q), np64(kp), np64(vp), np64(k), np64(v), lens, scale)
    close(got[0], Or, (U + F) * size + U * np.abs(Or), "O")
    empty = lr == -np.inf
    assert (np64(got[1])[empty] == -np.inf).all() and (np64(got[0])[empty] == 0).all()
    close(got[1][~torch.from_numpy(empty)], lr[~empty], 2 * F, "lse")


@pytest.mark.parametrize("case", PREFIX, ids=lambda c: "B{}H{}kv{}P{}S{}D{}".format(*c))
def test_prefix(case):
    B, H, Hkv, P, S, D, lens = case
    q, kp, vp, k, v = rand(61, B, H, D), rand(62, P, Hkv, D), rand(63, P, Hkv, D), rand(64, B, S, Hkv, D), rand(65, B, S, Hkv, D)
    kp[P // 2::5] *= 3                     # maxima that rise along the keys
    for b, n in enumerate(lens):
        k[b, n:], v[b, n:] = NAN, float("inf")
    ws = torch.full((dfa.dfa_attn_decode_prefix_workspace_size(B, H, Hkv, P, D),), 0xFF, dtype=torch.uint8, device=DEV)
    got = dfa.dfa_attn_decode_prefix(q, kp, vp, k, v, lens_of(lens), workspace_buf=ws)
    dfa.dfa_check_errors()
    check_prefix(got, q, kp, vp, k, v, lens)
    again = dfa.dfa_attn_decode_prefix(q, kp, vp, k, v, lens_of(lens))
    assert torch.equal(got[0], again[0]) and torch.equal(got[1], again[1])


def test_prefix_strides_lengths_out_of_range_and_scale():
    B, H, Hkv, P, S, D = 3, 4, 2, 200, 50, 128
    both = rand(71, Hkv, P, 2, D + 8)               # head-major, k and v interleaved
    kp, vp = both[..., 0, :D].transpose(0, 1), both[..., 1, :D].transpose(0, 1)
    own = rand(72, B, Hkv, S, 2, D + 8)
    k, v = own[..., 0, :D].transpose(1, 2), own[..., 1, :D].transpose(1, 2)
    q = rand(73, B, H, D)
    got = dfa.dfa_attn_decode_prefix(q, kp, vp, k, v, lens_of([-4, 20, 999]), scale=0.2)
    dfa.dfa_check_errors()
    check_prefix(got, q, kp, vp, k, v, [0, 20, 50], 0.2)


def test_prefix_is_the_step_over_a_cache_that_holds_it():
    B, H, Hkv, P, S, D = 12, 24, 3, 5000, 300, 128
    lens = [25 * i for i in range(B)]
    q, kp, vp, k, v = rand(74, B, H, D), rand(75, P, Hkv, D), rand(76, P, Hkv, D), rand(77, B, S, Hkv, D), rand(78, B, S, Hkv, D)
    O, lse = dfa.dfa_attn_decode_prefix(q, kp, vp, k, v, lens_of(lens))
    kk, vv = (torch.cat((t.expand(B, P, Hkv, D), own), 1) for t, own in ((kp, k), (vp, v)))
    want = dfa.dfa_attn_decode_sink(q, kk, vv, lens_of([P + n for n in lens]), P + S)
    dfa.dfa_check_errors()
    # both sides round P and the result; sum_j P |v_j| stays below 1.5
    assert (O.float() - want[0].float()).abs().max() <= 2 * (U + F) * 1.5 + 2 * U
    assert (lse - want[1]).abs().max() <= 4 * F


def test_prefix_of_nans_and_scores_below_32_bits():
    """As of the step: in the prefix and among the own keys; a CTA per segment, and parts that are joined."""
    for B, H, Hkv, P, S, D, lens in ((3, 8, 2, 500, 20, 64, [20, 0, 7]), (5, 12, 4, 700, 400, 128, [400, 0, 64, 7, 399])):
        q, kp, vp, k, v = rand(91, B, H, D), rand(92, P, Hkv, D), rand(93, P, Hkv, D), rand(94, B, S, Hkv, D), rand(95, B, S, Hkv, D)
        q[:, :, 0], kp[:, :, 0], k[:, :, :, 0] = 2.0 ** 100, 0, 0
        kp[:200, :, 0], k[:, :17, :, 0], k[:, 70:210, :, 0] = -2.0 ** 100, -2.0 ** 100, -2.0 ** 100
        n, G = lens_of(lens), H // Hkv
        got = dfa.dfa_attn_decode_prefix(q, kp, vp, k, v, n)
        dfa.dfa_check_errors()
        check_prefix(got, q, kp, vp, k, v, lens)
        bad = kp.clone()
        bad[P - 100, 1, 5] = NAN
        O, lse = dfa.dfa_attn_decode_prefix(q, bad, vp, k, v, n)
        assert O[:, G:2 * G].isnan().all() and lse[:, G:2 * G].isnan().all()
        others = torch.tensor([h for h in range(H) if h // G != 1], device=DEV)
        assert torch.equal(O[:, others], got[0][:, others]) and torch.equal(lse[:, others], got[1][:, others])
        bad = q.clone()
        bad[1, 0, 5] = NAN                     # of the sequence without own keys
        O, lse = dfa.dfa_attn_decode_prefix(bad, kp, vp, k, v, n)
        dfa.dfa_check_errors()
        assert O[1, 0].isnan().all() and lse[1, 0].isnan()
        O[1, 0], lse[1, 0] = got[0][1, 0], got[1][1, 0]
        assert torch.equal(O, got[0]) and torch.equal(lse, got[1])


def test_prefix_beyond_32_bits():
    B, H, Hkv, P, S, D = 2, 16, 8, (1 << 21) + 77, 10, 128
    kp, vp = (torch.empty(P, Hkv, D, dtype=torch.bfloat16, device=DEV).normal_(generator=gen(79 + i)) for i in range(2))
    q, k, v = rand(81, B, H, D), rand(82, B, S, Hkv, D), rand(83, B, S, Hkv, D)
    O, lse = dfa.dfa_attn_decode_prefix(q, kp, vp, k, v, lens_of([10, 0]))
    dfa.dfa_check_errors()
    s = [torch.einsum("hd,jd->hj", q[0, :2].double(), torch.cat((kp[:, 0], k[0, :, 0])).double()) * D ** -0.5,
         torch.einsum("hd,jd->hj", q[1, -2:].double(), kp[:, -1].double()) * D ** -0.5]
    vs = [torch.cat((vp[:, 0], v[0, :, 0])).double(), vp[:, -1].double()]
    for b, hs in ((0, slice(0, 2)), (1, slice(H - 2, H))):
        p = torch.softmax(s[b], -1)
        size, ref = np64(p @ vs[b].abs()), np64(p @ vs[b])
        close(O[b, hs], ref, (U + F) * size + U * np.abs(ref), "O")
        close(lse[b, hs], np64(torch.logsumexp(s[b], -1)), 2 * F, "lse")


# ------------------------------------------------------------------------------------------------ eviction
# (B, Hkv, S, D, keep, cap, n_first, n_recent, lens)
EVICT = [
    (1, 1, 1, 64, 1, 1, 0, 0, [1]), (2, 3, 5, 128, 3, 4, 1, 1, [0, 5]), (2, 2, 33, 64, 32, 40, 4, 8, [33, 32]),
    (1, 8, 501, 64, 128, 200, 4, 32, [501]), (3, 2, 1000, 128, 10, 10, 5, 5, [1000, 11, 10]), (2, 1, 1025, 64, 1024, 1024, 0, 0, [1025, 1024]),
    (2, 4, 2500, 128, 700, 701, 0, 100, [2500, 2049]), (1, 2, 9000, 64, 4000, 4500, 3, 0, [8999]), (2, 2, 40000, 64, 1000, 1000, 4, 64, [40000, 1001]),
    (1, 1, 70001, 128, 69999, 70001, 1, 1, [70001]), (1, 3, 131, 64, 300, 400, 7, 200, [131]), (5, 1, 64, 64, 1, 1, 0, 0, [64, 1, 0, 2, 63]),
]
EVICT_IDS = ["B{}kv{}S{}D{}k{}c{}f{}r{}".format(*c) for c in EVICT]


def check_evict(got, k, v, m, lens, case, behind=0):
    B, Hkv, S, D, keep, cap, n_first, n_recent, _ = case
    ko, vo, lo, mo, kept = got
    m = m.cpu().numpy()
    assert lo.tolist() == [min(n, keep) for n in lens]
    for b, n in enumerate(lens):
        for g in range(Hkv):
            j = cache.kept(m[b, g], n, keep, n_first, n_recent)
            assert kept[b, g].tolist() == j.tolist() + [-1] * (keep - len(j)), (b, g)
            at, r = torch.from_numpy(j).to(DEV), len(j)
            assert torch.equal(ko[b, :r, g], k[b, at, g]) and torch.equal(vo[b, :r, g], v[b, at, g]), (b, g)
            assert (ko[b, r:, g] == behind).all() and (vo[b, r:, g] == behind).all()
            assert np.array_equal(mo[b, g].cpu().numpy()[:r], m[b, g, j], equal_nan=True) and (mo[b, g, r:] == 0).all()


@pytest.mark.parametrize("kind", ["spread", "ties", "few", "odd"])
@pytest.mark.parametrize("case", EVICT, ids=EVICT_IDS)
def test_evict(case, kind):
    B, Hkv, S, D, keep, cap, n_first, n_recent, lens = case
    k, v = rand(31, B, S, Hkv, D), rand(32, B, S, Hkv, D)
    m = torch.exp(3 * rand(33, B, Hkv, S, dtype=torch.float32))
    if kind == "ties":                   # most of the masses equal, the border among them
        m = torch.where(m > 9, m, 0.0)
    elif kind == "few":                  # a handful of values, whole and of both signs
        m = (m * 2).clamp(max=6).round() - 3
    elif kind == "odd":                  # what a mass should not be, and what no order may stumble over
        for i, x in enumerate((NAN, float("inf"), -float("inf"), 0.0, -0.0, 1e-45, -1e-45, 3.4e38, -NAN)):
            m[..., i::17] = x
    for b, n in enumerate(lens):
        m[b, :, n:] = float("inf")       # behind the sequence: not a key
    ko, vo = (torch.full((B, cap, Hkv, D), 7, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    got = dfa.dfa_cache_evict(k, v, lens_of(lens), m, keep, n_first, n_recent, ko, vo)
    check_evict(got, k, v, m, lens, case, 7)
    again = dfa.dfa_cache_evict(k, v, lens_of(lens), m, keep, n_first, n_recent)
    check_evict(again, k, v, m, lens, (B, Hkv, S, D, keep, keep, n_first, n_recent, lens))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("S", [4093, 4094, 4095, 4096, 4097])
def test_evict_rows_that_do_not_begin_on_16_bytes(S, dtype):
    """The masses of a row are read 16 bytes at a time and a CTA's threads hold 4096 keys at once: rows that begin
    off 16 bytes, those of odd lengths and of a mass that is a slice, spill into a second turn.  Moved in one launch
    (few kept) and in two."""
    Hkv, D = 3, 64
    lens = [S, S - 1, S - 3]
    k, v = rand(35, 3, S, Hkv, D, dtype=dtype), rand(36, 3, S, Hkv, D, dtype=dtype)
    flat = torch.exp(3 * rand(37, 3 * Hkv * S + 3, dtype=torch.float32))
    for off in range(4):
        m = flat[off:off + 3 * Hkv * S].view(3, Hkv, S)
        for keep, n_first, n_recent in ((1, 0, 0), (64, 0, 63), (256, 0, 0), (200, 199, 0), (513, 0, 9)):
            ko, vo = (torch.full((3, keep + 1, Hkv, D), 7, dtype=dtype, device=DEV) for _ in range(2))
            got = dfa.dfa_cache_evict(k, v, lens_of(lens), m, keep, n_first, n_recent, ko, vo)
            dfa.dfa_check_errors()
            check_evict(got, k, v, m, lens, (3, Hkv, S, D, keep, keep + 1, n_first, n_recent, lens), 7)


@pytest.mark.parametrize("S", [16384, 32767, 65536, 131071, 131073])
def test_evict_long_rows_that_do_not_begin_on_16_bytes(S):
    """The same where a CTA, two, four or eight of a cluster hold a row but for the keys that its misalignment pushes out."""
    Hkv, D, keep = 2, 64, 700
    k, v = rand(38, 1, S, Hkv, D), rand(39, 1, S, Hkv, D)
    flat = torch.exp(3 * rand(40, Hkv * S + 3, dtype=torch.float32)).clamp(max=50)      # the border among equal ones
    for off in (0, 1, 3):
        m = flat[off:off + Hkv * S].view(1, Hkv, S)
        ko, vo = (torch.full((1, keep, Hkv, D), 7, dtype=torch.bfloat16, device=DEV) for _ in range(2))
        got = dfa.dfa_cache_evict(k, v, lens_of([S]), m, keep, 2, 9, ko, vo)
        dfa.dfa_check_errors()
        check_evict(got, k, v, m, [S], (1, Hkv, S, D, keep, keep, 2, 9, [S]), 7)


def test_evict_strides_types_and_lengths_out_of_range():
    B, Hkv, S, D, keep, cap = 3, 2, 300, 128, 50, 60
    lens = [0, 250, 300]
    m = rand(41, B, Hkv, S, dtype=torch.float32)
    n = lens_of([-7, 250, 1000])
    both = rand(42, B, Hkv, S, 2, D + 8)                            # head-major, k and v interleaved
    k, v = both[..., 0, :D].transpose(1, 2), both[..., 1, :D].transpose(1, 2)
    out = torch.full((B, Hkv, cap, 2, D + 8), 7.0, device=DEV).bfloat16()
    ko, vo = out[..., 0, :D].transpose(1, 2), out[..., 1, :D].transpose(1, 2)
    case = (B, Hkv, S, D, keep, cap, 2, 9, lens)
    check_evict(dfa.dfa_cache_evict(k, v, n, m, keep, 2, 9, ko, vo), k, v, m, lens, case, 7)
    assert (out[..., D:] == 7).all()
    k, v = rand(43, B, S, Hkv, D, dtype=torch.float32), rand(44, B, S, Hkv, D, dtype=torch.float32)
    ko, vo = (torch.full((B, cap, Hkv, D), 7.0, device=DEV) for _ in range(2))
    check_evict(dfa.dfa_cache_evict(k, v, n, m, keep, 2, 9, ko, vo), k, v, m, lens, case, 7)
    shared = rand(45, 1, S, Hkv, D).expand(B, S, Hkv, D)            # one cache for the batch: a stride of 0
    check_evict(dfa.dfa_cache_evict(shared, shared, n, m, keep, 2, 9), shared, shared, m, lens, (B, Hkv, S, D, keep, keep, 2, 9, lens))


def test_evict_into_two_slices_of_one_buffer():
    """k_out and v_out side by side, whatever dimension they share; none of these has a common element."""
    B, Hkv, S, D, keep, cap = 2, 2, 200, 64, 30, 32
    k, v, m = rand(49, B, S, Hkv, D), rand(50, B, S, Hkv, D), rand(51, B, Hkv, S, dtype=torch.float32)
    lens = [200, 20]
    pool = lambda *s: torch.full(s, 7, dtype=torch.bfloat16, device=DEV)  # noqa: E731
    pairs = [(x[:, :cap], x[:, cap:]) for x in [pool(B, 2 * cap, Hkv, D)]] + [(x[:, ::2], x[:, 1::2]) for x in [pool(B, 2 * cap, Hkv, D)]] + \
        [(x[:, :, ::2], x[:, :, 1::2]) for x in [pool(B, cap, 2 * Hkv, D)]] + [(x[..., :D], x[..., D:]) for x in [pool(B, cap, Hkv, 2 * D)]] + \
        [(x[:B], x[B:]) for x in [pool(2 * B, cap, Hkv, D)]] + [(x[::2], x[1::2]) for x in [pool(2 * B, cap, Hkv, D)]] + \
        [(x[:, 0:2 * cap:2], x[:, 5:5 + 2 * cap:2]) for x in [pool(B, 2 * cap + 5, Hkv, D)]] + \
        [(x[:, 1].permute(1, 2, 0, 3), x[:, 0].permute(1, 2, 0, 3)) for x in [pool(Hkv, 2, B, cap, D)]]
    for ko, vo in pairs:
        got = dfa.dfa_cache_evict(k, v, lens_of(lens), m, keep, 2, 3, ko, vo)
        check_evict(got, k, v, m, lens, (B, Hkv, S, D, keep, cap, 2, 3, lens), 7)
    x = pool(B, 2 * cap, Hkv, D)
    for ko, vo in ((x[:, :cap], x[:, cap - 1:-1]), (x[:, ::2], x[:, ::2]), (x[:, 4:4 + cap], x[:, 1:1 + cap])):
        with pytest.raises(dfa.DfaError, match="same memory"):
            dfa.dfa_cache_evict(k, v, lens_of(lens), m, keep, 2, 3, ko, vo)
    assert (x == 7).all()
    dfa.dfa_check_errors()


def test_evict_from_a_cache_beyond_32_bits():
    B, Hkv, S, D, keep = 3, 8, (1 << 20) + 5, 128, 300
    k, v = (torch.empty(B, S, Hkv, D, dtype=torch.bfloat16, device=DEV).normal_(generator=gen(46 + i)) for i in range(2))
    m = torch.rand(B, Hkv, S, device=DEV, generator=gen(48))
    lens = [S, 17, S - 1]
    ko, vo, lo, mo, kept = dfa.dfa_cache_evict(k, v, lens_of(lens), m, keep, 4, 16)
    for b, n in enumerate(lens):
        r = min(n, keep)
        for g in range(Hkv):
            at = kept[b, g, :r].long()
            if n > keep:
                top = torch.topk(m[b, g, 4:n - 16], keep - 20).indices + 4
                want = torch.cat((torch.arange(4, device=DEV), top.sort().values, torch.arange(n - 16, n, device=DEV)))
                assert torch.equal(m[b, g, at].sort().values, m[b, g, want].sort().values) and (at[1:] > at[:-1]).all()
            assert torch.equal(ko[b, :r, g], k[b, at, g]) and torch.equal(vo[b, :r, g], v[b, at, g])
            assert torch.equal(mo[b, g, :r], m[b, g, at])


# ------------------------------------------------------------------------------------------------ together
def test_a_prompt_evicted_continued_and_evicted_again():
    """A prompt's forward, its masses, a smaller cache, tokens through one captured step that adds to the masses, the
    cache cut down again: each step against the reference on what the cache holds then."""
    B, H, Hkv, D, S, keep, cap = 2, 8, 2, 128, 900, 300, 340
    q, k, v = rand(91, B, S + 60, H, D), rand(92, B, S + 60, Hkv, D), rand(93, B, S + 60, Hkv, D)
    O, lse = dfa.dfa_attn_fwd(q[:, :S].contiguous(), k[:, :S].contiguous(), v[:, :S].contiguous())
    m = dfa.dfa_attn_mass(q[:, :S].contiguous(), k[:, :S].contiguous(), lse)
    close(m, cache.mass(np64(q[:, :S]), np64(k[:, :S]), np64(lse), S, 0, S), 2 * F * np64(m), "mass")
    kc, vc = (torch.full((B, cap, Hkv, D), NAN, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    _, _, n, mc, kept = dfa.dfa_cache_evict(k[:, :S], v[:, :S], lens_of([S, S]), m, keep, 4, 50, kc, vc)
    held = [[[int(j) for j in kept[b, g]] for g in range(Hkv)] for b in range(B)]
    qt = torch.empty(B, H, D, dtype=torch.bfloat16, device=DEV)

    def capture(kc, vc, n, mc):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = dfa.dfa_attn_decode_mass(qt, kc, vc, n, mc, mass_out=mc)
        return graph, out

    def follow(i, graph, out, kc, vc, n, mc):
        at = n.clone()
        for b in range(B):
            kc[b, at[b]], vc[b, at[b]] = k[b, i], v[b, i]
            for g in range(Hkv):
                held[b][g].append(i)
        qt.copy_(q[:, i])
        n.add_(1)
        before = np64(mc)
        graph.replay()
        for b in range(B):
            for h in range(H):
                g = h * Hkv // H
                j = torch.tensor(held[b][g], device=DEV)
                Or, lr, size = sink.decode(np64(qt[b:b + 1, h:h + 1]), np64(k[b:b + 1, j][:, :, g:g + 1]), np64(v[b:b + 1, j][:, :, g:g + 1]),
                                           [len(j)], len(j), 0)
                close(out[0][b:b + 1, h:h + 1], Or, (U + F) * size + U * np.abs(Or), "O")
                close(out[1][b:b + 1, h:h + 1], lr, 2 * F, "lse")
        np.testing.assert_allclose(np64(mc).sum((1, 2)) - before.sum((1, 2)), H, rtol=1e-2)
        return int(n[0])

    graph, out = capture(kc, vc, n, mc)
    for i in range(S, S + 40):
        last = follow(i, graph, out, kc, vc, n, mc)
    assert last == cap
    k2, v2 = (torch.full((B, cap, Hkv, D), NAN, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    masses = mc.clone()
    _, _, n2, m2, kept2 = dfa.dfa_cache_evict(kc, vc, n, mc, 100, 4, 20, k2, v2)
    for b in range(B):
        for g in range(Hkv):
            assert kept2[b, g].tolist() == cache.kept(masses[b, g].cpu().numpy(), cap, 100, 4, 20).tolist()
            held[b][g] = [held[b][g][j] for j in kept2[b, g].tolist()]
    graph2, out2 = capture(k2, v2, n2, m2)
    for i in range(S + 40, S + 50):
        follow(i, graph2, out2, k2, v2, n2, m2)
    dfa.dfa_check_errors()


def everything(stream=None, seed=101):
    """One call of each kind: small ones that run in clusters or one CTA, large ones that are cut."""
    got = []
    for B, H, Hkv, S, D, window, N, last in ((1, 4, 2, 700, 64, 700, 0, 700), (2, 8, 4, 2600, 128, 900, 3, 2600), (1, 4, 2, 3000, 128, 3000, 0, 40)):
        q, k, lse = rand(seed, B, S, H, D), rand(seed + 1, B, S, Hkv, D), rand(seed + 2, B, H, S, dtype=torch.float32) + 8
        got.append(dfa.dfa_attn_mass(q, k, lse, window, N, last, stream=stream))
    for B, H, Hkv, S, D, lens in ((1, 8, 4, 900, 128, [801]), (9, 16, 8, 2500, 64, [i * 300 for i in range(9)])):
        q, k, v, m = rand(seed + 3, B, H, D), rand(seed + 4, B, S, Hkv, D), rand(seed + 5, B, S, Hkv, D), rand(seed + 6, B, Hkv, S, dtype=torch.float32).abs()
        got += dfa.dfa_attn_decode_mass(q, k, v, lens_of(lens), m, stream=stream)
        for keep in (64, 700):
            got += dfa.dfa_cache_evict(k, v, lens_of(lens), m, keep, 2, 30, stream=stream)
        for P in (0, 90, 2000):
            kp, vp = rand(seed + 7, P, Hkv, D), rand(seed + 8, P, Hkv, D)
            got += dfa.dfa_attn_decode_prefix(q, kp, vp, k, v, lens_of(lens), stream=stream)
            got += dfa.dfa_attn_decode_prefix(q, kp, vp, k[:, :100].contiguous(), v[:, :100].contiguous(), lens_of(lens), stream=stream)
    return got


def same(a, b):
    return len(a) == len(b) and all(torch.equal(x, y) for x, y in zip(a, b))


def test_the_same_bits_on_every_call_and_from_a_graph(monkeypatch):
    want = everything()
    assert same(everything(), want)
    # the inputs are made outside the graph: what makes them is not captured
    made = {}
    for name in ("rand", "lens_of"):
        def once(*a, make=globals()[name], **kw):
            key = str((make, a, kw))
            if key not in made:
                made[key] = make(*a, **kw)
            return made[key]
        monkeypatch.setitem(globals(), name, once)
    everything()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = everything()
    for _ in range(2):
        for t in got:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert same(got, want)
    dfa.dfa_check_errors()


def test_calls_on_other_streams_and_from_threads():
    import threading
    want = [everything(seed=s) for s in (111, 131)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in want]
    for _ in range(3):
        got = []
        for st, seed in zip(streams, (111, 131)):
            st.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(st):
                got.append(everything(seed=seed))
        torch.cuda.synchronize()
        assert all(same(a, b) for a, b in zip(got, want))
    failed = []

    def work(i):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for _ in range(5):
                    assert same(everything(seed=(111, 131)[i % 2]), want[i % 2])
        except BaseException as e:       # shown by the test, not lost with the thread
            failed.append(e)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    dfa.dfa_check_errors()
    assert not failed, failed


def test_a_call_on_another_stream_holds_its_tensors():
    """Inputs dropped while the other stream has still to read them, outputs from memory that the current stream is about
    to write."""
    B, H, Hkv, S, D = 2, 8, 2, 1200, 128
    s = torch.cuda.Stream()

    def made():
        return (rand(141, B, H, D), rand(142, 300, Hkv, D), rand(143, 300, Hkv, D), rand(144, B, S, Hkv, D), rand(145, B, S, Hkv, D),
                lens_of([1200, 700]), rand(146, B, Hkv, S, dtype=torch.float32).abs(), rand(147, B, S, H, D), rand(148, B, H, S, dtype=torch.float32) + 8)

    def calls(q, kp, vp, k, v, n, m, qs, lse, stream=None):
        return [dfa.dfa_attn_mass(qs, k, lse, stream=stream)] + list(dfa.dfa_attn_decode_mass(q, k, v, n, m, stream=stream)) + \
            list(dfa.dfa_cache_evict(k, v, n, m, 800, 3, 40, stream=stream)) + list(dfa.dfa_attn_decode_prefix(q, kp, vp, k, v, n, stream=stream))

    want = calls(*made())
    for _ in range(3):
        data = made()
        torch.cuda.synchronize()
        blocks = [torch.empty_like(t) for t in want]
        torch.cuda._sleep(20000000)
        for t in blocks:
            t.fill_(7)
        del blocks
        with torch.cuda.stream(s):
            torch.cuda._sleep(20000000)
        got = calls(*data, stream=s)
        sizes = [torch.empty_like(t, device="meta") for t in data]
        del data
        fill = [torch.full_like(t, 1, device=DEV) for t in sizes]
        torch.cuda.synchronize()
        assert same(got, want)
        del fill
    dfa.dfa_check_errors()


def test_workspaces_go_back_and_outputs_are_ordinary_tensors():
    """Calls leave no memory behind, refused ones and those on another stream neither; in inference mode the outputs are
    what torch makes there."""
    want, s = everything(), torch.cuda.Stream()
    q, k = rand(1, 2, 4, 64), rand(2, 2, 40, 2, 64)
    n, m = lens_of([9, 9]), torch.zeros(2, 2, 40, device=DEV)
    torch.cuda.synchronize()
    before = torch.cuda.memory_allocated()
    for _ in range(3):
        got = everything()
        assert same(got, want)
        del got
        with pytest.raises(dfa.DfaError):
            dfa.dfa_attn_decode_mass(q, k, k, n, m, window=0)
        del _
        dfa.dfa_attn_decode_prefix(q, k[0], k[0], k, k, n, stream=s)
        torch.cuda.synchronize()
        assert torch.cuda.memory_allocated() == before
    with torch.inference_mode():
        got = everything()
        assert all(t.is_inference() for t in got) and same(got, want)
    assert not any(t.is_inference() or t.requires_grad for t in want)
    dfa.dfa_check_errors()


FIRST = """
import torch
from long_context_causal_gb300 import dfa
g = torch.Generator("cuda").manual_seed(1)
r = lambda *s: torch.randn(*s, device="cuda", generator=g).bfloat16()
for D in (64, 128):
    q, k, v, qs, kp, vp = r(2, 8, D), r(2, 600, 2, D), r(2, 600, 2, D), r(2, 600, 8, D), r(200, 2, D), r(200, 2, D)
    n, m, lse = torch.full((2,), 555, dtype=torch.int32, device="cuda"), torch.rand(2, 2, 600, device="cuda"), torch.full((2, 8, 600), 9.0, device="cuda")
    chain = lambda: (dfa.dfa_attn_mass(qs, k, lse), dfa.dfa_attn_mass(qs, k, lse, n_last=30)) + dfa.dfa_attn_decode_mass(q, k, v, n, m) + \\
        dfa.dfa_cache_evict(k, v, n, m, 100) + dfa.dfa_attn_decode_prefix(q, kp, vp, k, v, n)
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
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", FIRST], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]


def test_mass_beyond_32_bits():
    """2^31 elements in q: keys of the last head and the end of the sequence."""
    B, H, Hkv, S, D, W, N = 1, 32, 8, 524288 + 77, 128, 300, 4
    q, k = (torch.empty(B, S, h, D, dtype=torch.bfloat16, device=DEV).normal_(generator=gen(151 + h)) for h in (H, Hkv))
    lse = torch.rand(B, H, S, device=DEV, generator=gen(152)) + 6
    for n_last in (S, 50):
        m = dfa.dfa_attn_mass(q, k, lse, W, N, n_last)
        dfa.dfa_check_errors()
        for j in (S - 1, S - 60, S - 349, S - 700, 2):
            i = torch.arange(max(j, S - n_last), S if j < N else max(min(j + W, S), max(j, S - n_last)), device=DEV)
            s = torch.einsum("ihd,hd->hi", q[0, i].double(), k[0, j].double().repeat_interleave(H // Hkv, 0)) * D ** -0.5
            w = torch.exp(s - lse[0][:, i].double()).sum(1).reshape(Hkv, -1).sum(1)
            # sums of up to 2^12 tiles of 128: as many additions in fp32
            close(m[0, :, j], np64(w), (F + 2.0 ** -12) * np64(w), "mass")


def test_empty_batches_and_no_tokens():
    H, Hkv, D = 4, 2, 64
    t = lambda *s, dtype=torch.bfloat16: torch.zeros(s, dtype=dtype, device=DEV)  # noqa: E731
    for B, S in ((0, 50), (3, 0)):
        assert dfa.dfa_attn_mass(t(B, S, H, D), t(B, S, Hkv, D), t(B, H, S, dtype=torch.float32)).shape == (B, Hkv, S)
    q, k, n, m = t(0, H, D), t(0, 9, Hkv, D), t(0, dtype=torch.int32), t(0, Hkv, 9, dtype=torch.float32)
    assert [x.shape for x in dfa.dfa_attn_decode_mass(q, k, k, n, m)] == [(0, H, D), (0, H), (0, Hkv, 9)]
    assert [x.shape[0] for x in dfa.dfa_cache_evict(k, k, n, m, 4)] == [0] * 5
    assert [x.shape for x in dfa.dfa_attn_decode_prefix(q, t(5, Hkv, D), t(5, Hkv, D), k, k, n)] == [(0, H, D), (0, H)]
    with pytest.raises(dfa.DfaError, match="room"):
        dfa.dfa_attn_decode_mass(t(2, H, D), t(2, 0, Hkv, D), t(2, 0, Hkv, D), t(2, dtype=torch.int32))
    dfa.dfa_check_errors()


def test_what_the_binding_refuses_on_the_gpu():
    B, H, Hkv, S, D = 2, 4, 2, 40, 64
    q, k, n, m = rand(1, B, H, D), rand(2, B, S, Hkv, D), lens_of([9, 9]), torch.zeros(B, Hkv, S, device=DEV)
    with pytest.raises(dfa.DfaError, match="overlaps"):
        dfa.dfa_cache_evict(k, k.clone(), n, m, 10, k_out=k[:, :20], v_out=k[:, 20:])
    with pytest.raises(dfa.DfaError, match="overlaps"):
        dfa.dfa_cache_evict(k, k, n, m, 10, len_out=n)
    with pytest.raises(dfa.DfaError, match="same memory"):
        x = k.clone()
        dfa.dfa_cache_evict(k, k, n, m, 10, k_out=x, v_out=x)
    with pytest.raises(ValueError, match="together"):
        dfa.dfa_cache_evict(k, k, n, m, 10, k_out=k.clone())
    with pytest.raises(ValueError, match="caches of k"):
        dfa.dfa_cache_evict(k, k, n, m, 10, k_out=k.float(), v_out=k.float())
    with pytest.raises(dfa.DfaError, match="cap"):
        dfa.dfa_cache_evict(k, k, n, m, 10, k_out=rand(3, B, 9, Hkv, D), v_out=rand(4, B, 9, Hkv, D))
    for bad in ((0, 0, 0), (10, 6, 5), (10, -1, 0)):
        with pytest.raises((dfa.DfaError, ValueError)):
            dfa.dfa_cache_evict(k, k, n, m, *bad)
    with pytest.raises(ValueError, match="32-bit"):
        dfa.dfa_cache_evict(k, k, n, m, 1 << 31)
    with pytest.raises(ValueError, match="mass must be"):
        dfa.dfa_attn_decode_mass(q, k, k, n, m[:, :, :-1].contiguous())
    with pytest.raises(ValueError, match="kv_len must be"):
        dfa.dfa_attn_decode_mass(q, k, k, n.long(), m)
    with pytest.raises(dfa.DfaError):
        dfa.dfa_attn_decode_mass(q.float(), k.float(), k.float(), n, m)
    with pytest.raises(dfa.DfaError, match="broadcast"):
        dfa.dfa_attn_decode_prefix(q, rand(5, 1, Hkv, D).expand(7, Hkv, D), rand(6, 1, Hkv, D).expand(7, Hkv, D), k, k, n)
    with pytest.raises(ValueError, match="workspace"):
        dfa.dfa_attn_decode_prefix(q, k[0], k[0], k, k, n, workspace_buf=torch.zeros(9, device=DEV))
    with pytest.raises(dfa.DfaError, match="workspace"):
        dfa.dfa_attn_mass(rand(7, B, S, H, D), k, torch.zeros(B, H, S, device=DEV), workspace_buf=torch.zeros(16, dtype=torch.uint8, device=DEV))
    with pytest.raises(dfa.DfaError, match="n_last"):
        dfa.dfa_attn_mass(rand(7, B, S, H, D), k, torch.zeros(B, H, S, device=DEV), n_last=0)
    assert dfa.dfa_attn_mass(rand(7, B, S, H, D), k, torch.zeros(B, H, S, device=DEV), n_last=1 << 30).shape == (B, Hkv, S)
    dfa.dfa_check_errors()


def test_a_stream_of_another_device_is_refused_by_the_binding():
    """By every call that it marshals, before anything is allocated or launched (a stand-in: there may be one device)."""
    class Elsewhere:
        device_index, cuda_stream = torch.cuda.current_device() + 1, torch.cuda.current_stream().cuda_stream

    class Here:
        device_index, cuda_stream = torch.cuda.current_device(), torch.cuda.current_stream().cuda_stream

    B, H, Hkv, S, D = 2, 4, 2, 40, 64
    q, k, n, m, qs, lse = rand(1, B, H, D), rand(2, B, S, Hkv, D), lens_of([9, 9]), torch.zeros(B, Hkv, S, device=DEV), rand(3, B, S, H, D), torch.zeros(B, H, S, device=DEV)
    kept = dfa.dfa_ckpt8_save(qs, k, k, qs)
    calls = [lambda s: dfa.dfa_attn_mass(qs, k, lse, stream=s), lambda s: dfa.dfa_attn_decode_mass(q, k, k, n, m, stream=s),
             lambda s: dfa.dfa_cache_evict(k, k, n, m, 10, stream=s), lambda s: dfa.dfa_attn_decode_prefix(q, k[0], k[0], k, k, n, stream=s),
             lambda s: dfa.dfa_attn_decode_sink(q, k, k, n, 8, stream=s), lambda s: dfa.dfa_attn_fwd_sink(qs, k, k, 8, stream=s),
             lambda s: dfa.dfa_attn_bwd_sink(qs, k, k, qs, lse, qs, 8, stream=s), lambda s: dfa.dfa_ckpt8_save(qs, k, k, qs, stream=s),
             lambda s: dfa.dfa_ckpt8_restore(kept, B, S, H, Hkv, D, stream=s), lambda s: dfa.dfa_attn_bwd_ckpt8(kept, lse, qs, Hkv, 8, stream=s)]
    torch.cuda.synchronize()
    before = torch.cuda.memory_allocated()
    for call in calls:
        with pytest.raises(ValueError, match="the stream is on cuda:"):
            call(Elsewhere)
    assert torch.cuda.memory_allocated() == before
    for s in (Here, torch.cuda.current_stream(), Here.cuda_stream, torch.cuda.Stream()):
        assert torch.equal(calls[0](s), calls[0](None))
        torch.cuda.synchronize()
    dfa.dfa_check_errors()
