"""Serving from a long cache, as it is measured: attention weights gathered per key, eviction by them, a shared prefix.

Four kinds of case:
  mass    over a prompt: the attention weight that each key of each key/value head drew from the last `n_last` queries
          (all of them: what the prompt's eviction looks at; a few: an observation window at its end)
  step    one new token per sequence over a cache: O and lse, and its weights added to the keys' masses
  evict   the `keep` keys of each sequence and head with the greatest mass, the first and the last ones among them in
          any case, moved in their order to a smaller cache
  prefix  one new token per sequence where all sequences share their first tokens' keys and values

With `own` False, `run` computes them with elementary torch operations in 32 bits; with `own` True it makes the
library's calls.  Shapes: q [B, S, H, D] (one token: [B, H, D]), k, v [B, S, Hkv, D] and prefixes [P, Hkv, D] in bf16;
lse [B, H, S], mass [B, Hkv, S] in fp32; lengths and kept positions int32.  Query head h reads head h / (H / Hkv).
"""
import math

import torch

own = False

DEV = "cuda"
PAIRS_MAX = 32768 * (4096 + 256) * 32       # score elements of the largest listed mass case's band
CACHE_MAX = 32 * 16384 * 8 * 128            # elements of the largest listed cache
PREFIX_MAX = 128 * 64 * 16384 * 128         # B H P D of the largest listed prefix case


# ------------------------------------------------------------------------------------------------ cases
def listed():
    return [
        # short prompts of a small model: the call's latency counts
        dict(name="mass short", kind="mass", B=2, S=301, H=4, Hkv=2, D=64, window=301, n_sink=0, n_last=301),
        # the observation window at the end of a 32K prompt
        dict(name="mass tail", kind="mass", B=1, S=32768, H=32, Hkv=8, D=128, window=32768, n_sink=0, n_last=64),
        # a batch of ragged length, plain causal, all queries
        dict(name="mass ragged batch", kind="mass", B=2, S=5003, H=16, Hkv=2, D=128, window=5003, n_sink=0, n_last=5003),
        # all queries of a 32K prompt under a window with sinks
        dict(name="mass 32K", kind="mass", B=1, S=32768, H=32, Hkv=8, D=128, window=4096, n_sink=4, n_last=32768),
        # a single user's next token over a cache that was cut down before
        dict(name="step one", kind="step", B=1, S=2048, H=32, Hkv=8, D=128, window=2048, n_sink=0, lo=1501, hi=1501),
        # a server's batch of next tokens, caches of all lengths
        dict(name="step batch", kind="step", B=32, S=16384, H=32, Hkv=8, D=128, window=16384, n_sink=0, lo=1, hi=16384),
        # a short prompt's cache, small head dim
        dict(name="evict small", kind="evict", B=1, S=501, Hkv=8, D=64, keep=128, cap=256, n_first=4, n_recent=32, lo=501, hi=501),
        # a batch of 16K caches, some of them short enough to keep whole, cut to a quarter
        dict(name="evict batch", kind="evict", B=8, S=16384, Hkv=8, D=128, keep=4096, cap=4608, n_first=4, n_recent=512, lo=3000, hi=16384),
        # one 128K prompt cut to an eighth
        dict(name="evict 128K", kind="evict", B=1, S=131072, Hkv=8, D=128, keep=16384, cap=16896, n_first=4, n_recent=1024, lo=131072, hi=131072),
        # four short continuations of one prompt
        dict(name="prefix few", kind="prefix", B=4, P=1000, S=64, H=32, Hkv=8, D=128, lo=1, hi=50),
        # a batch behind one 32K document
        dict(name="prefix batch", kind="prefix", B=48, P=32768, S=512, H=32, Hkv=8, D=128, lo=1, hi=512),
        # many samples of one problem, eight query heads per key/value head
        dict(name="prefix wide", kind="prefix", B=128, P=16384, S=1024, H=64, Hkv=8, D=128, lo=0, hi=1024),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    kind = rng.choice(["mass", "step", "evict", "prefix"])
    D = rng.choice([64, 128])
    Hkv = rng.choice([1, 2, 4, 8])
    H = Hkv * rng.choice([1, 2, 3, 4, 8])
    if kind == "mass":
        B, S = rng.choice([1, 1, 2, 3]), _log(rng, 1, 65536)
        window, n_sink = rng.choice([S, _log(rng, 1, S)]), rng.choice([0, 1, 4, 33, 128])
        n_last = rng.choice([S, _log(rng, 1, S)])
        while B * H * n_last * (min(window, S) + 256) > PAIRS_MAX // 2:
            S = S * 3 // 4
            window, n_last = min(window, S), min(n_last, S)
        return dict(kind=kind, B=B, S=S, H=H, Hkv=Hkv, D=D, window=window, n_sink=n_sink, n_last=n_last)
    if kind == "prefix":
        B, P, S = _log(rng, 1, 128), _log(rng, 1, 65536), _log(rng, 1, 2048)
        while B * H * P * D > PREFIX_MAX // 2:
            P = P * 3 // 4
        hi = rng.randint(0, S)
        return dict(kind=kind, B=B, P=P, S=S, H=H, Hkv=Hkv, D=D, lo=rng.randint(0, hi), hi=hi)
    B, S = _log(rng, 1, 32), _log(rng, 1, 131072)
    while B * S * Hkv * D > CACHE_MAX // 2:
        B = max(1, B // 2)
        S = S if B > 1 else S * 3 // 4
    hi = rng.randint(1, S)
    lo = rng.randint(0, hi)
    if kind == "step":
        return dict(kind=kind, B=B, S=S, H=H, Hkv=Hkv, D=D, window=rng.choice([S, _log(rng, 1, S)]),
                    n_sink=rng.choice([0, 1, 4, 17, 128]), lo=lo, hi=hi)
    keep = _log(rng, 1, S)
    n_first = rng.randint(0, min(keep, 8))
    return dict(kind=kind, B=B, S=S, Hkv=Hkv, D=D, keep=keep, cap=keep + rng.choice([0, 1, 512]), n_first=n_first,
                n_recent=rng.randint(0, (keep - n_first) // 2), lo=lo, hi=hi)


def _lens(case):
    n = case["B"]
    return [case["lo"] + (case["hi"] - case["lo"]) * b // max(n - 1, 1) for b in range(n)]


def work(case):
    kind, B, S, Hkv, D = (case[x] for x in ("kind", "B", "S", "Hkv", "D"))
    if kind == "evict":                       # the kept rows read and written, the masses read, what is kept told
        rows = sum(min(n, case["keep"]) for n in _lens(case)) * Hkv
        return {"bytes": 8 * rows * D + 4 * Hkv * sum(_lens(case)) + 4 * rows + 4 * B * Hkv * (case["cap"] + case["keep"]), "flops": 0}
    H = case["H"]
    if kind == "prefix":
        keys, own_keys = case["P"], sum(_lens(case))
        return {"bytes": 4 * (keys + own_keys) * Hkv * D + 4 * B * H * D + 4 * B * H + 4 * B, "flops": 4 * D * H * (B * keys + own_keys)}
    w, ns = min(case["window"], S), case["n_sink"]
    if kind == "step":
        keys = sum(min(n, w) + min(ns, max(n - w, 0)) for n in _lens(case))
        mass = 4 * Hkv * sum(_lens(case)) + 4 * B * Hkv * S
        return {"bytes": 4 * keys * Hkv * D + 4 * B * H * D + 4 * B * H + 4 * B + mass, "flops": 4 * D * H * keys}
    n = case["n_last"]
    pairs = sum(min(i + 1, w) + min(ns, max(i + 1 - w, 0)) for i in range(S - n, S))
    keys = min(S, n - 1 + w) + min(ns, max(S - n + 1 - w, 0))
    return {"bytes": B * (2 * n * H * D + 2 * keys * Hkv * D + 4 * H * n + 4 * Hkv * S), "flops": 2 * D * B * H * pairs}


# ------------------------------------------------------------------------------------------------ inputs
def prepare(case, seed):
    """Unit-normal activations; every thirtieth key (and the sinks, whose values are small) lies along the direction
    that all queries share and draws several times an ordinary key's weight.  Masses handed in are what such keys have
    gathered: spread over orders of magnitude, a fifth of them zero (keys that no query has seen yet)."""
    kind, B, S, Hkv, D = (case[x] for x in ("kind", "B", "S", "Hkv", "D"))
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    rnd = lambda *shape: torch.randn(shape, generator=gen, device=DEV)  # noqa: E731
    bf = lambda t: t.to(torch.bfloat16)  # noqa: E731
    u = rnd(Hkv, D)

    def keys(*shape):
        k = torch.empty(shape, dtype=torch.bfloat16, device=DEV)
        for part in k.split(max(1, (1 << 28) // max(1, k[0].numel()))):
            x = rnd(*part.shape)
            x.view(-1, *shape[-3:])[:, ::30] += u
            part.copy_(x)
        return k

    state = dict(case, scale=D ** -0.5)
    if kind in ("step", "evict", "prefix"):
        state["kv_len"] = torch.tensor(_lens(case), dtype=torch.int32, device=DEV)
        state["k"], state["v"] = keys(B, S, Hkv, D), keys(B, S, Hkv, D)
    if kind in ("step", "evict"):
        mass = torch.exp(2 * rnd(B, Hkv, S)) * (torch.rand(B, Hkv, S, generator=gen, device=DEV) > 0.2)
        live = torch.arange(S, device=DEV) < state["kv_len"][:, None, None]
        state["mass"] = torch.where(live, mass, 0.0)
    if kind == "evict":
        for name in ("k_out", "v_out"):       # the smaller cache, which the next tokens fill up
            state[name] = torch.zeros(B, case["cap"], Hkv, D, dtype=torch.bfloat16, device=DEV)
        return state
    H = case["H"]
    q = rnd(B, S if kind == "mass" else 1, H, D) + 0.25 * u.repeat_interleave(H // Hkv, 0)
    state["q"] = bf(q if kind == "mass" else q[:, 0])
    if kind == "prefix":
        state["k_prefix"], state["v_prefix"] = keys(1, case["P"], Hkv, D)[0], keys(1, case["P"], Hkv, D)[0]
    if kind == "mass":
        state["k"] = keys(B, S, Hkv, D)
        state["k"][:, :case["n_sink"]] = bf(0.3 * state["k"][:, :case["n_sink"]].float() + 1.5 * u)
        state["lse"] = torch.empty(B, H, S, device=DEV)
        for a, b, idx, seen in _blocks(state, 0):
            s = _scores(state, a, b, idx, seen)
            state["lse"][:, :, a:b] = torch.logsumexp(s, -1).reshape(B, H, b - a)
    return state


# ------------------------------------------------------------------------------------------------ one pass
def run(state):
    s = state
    if own:
        return _own(s)
    return {"mass": _plain_mass, "step": _plain_step, "evict": _plain_evict, "prefix": _plain_prefix}[s["kind"]](s)


def _own(s):
    from long_context_causal_gb300 import dfa
    if s["kind"] == "mass":
        return dfa.dfa_attn_mass(s["q"], s["k"], s["lse"], s["window"], s["n_sink"], s["n_last"], scale=s["scale"])
    if s["kind"] == "step":
        return dfa.dfa_attn_decode_mass(s["q"], s["k"], s["v"], s["kv_len"], s["mass"], s["window"], s["n_sink"], scale=s["scale"])
    if s["kind"] == "evict":
        return dfa.dfa_cache_evict(s["k"], s["v"], s["kv_len"], s["mass"], s["keep"], s["n_first"], s["n_recent"],
                                   k_out=s["k_out"], v_out=s["v_out"])
    return dfa.dfa_attn_decode_prefix(s["q"], s["k_prefix"], s["v_prefix"], s["k"], s["v"], s["kv_len"], scale=s["scale"])


# ------------------------------------------------------------------------------------------------ plain forms
def _blocks(s, first):
    """Rows [first, S) in blocks: (a, b, the positions of the keys that rows a .. b - 1 see, which of them each sees)."""
    S, w, ns = s["S"], min(s["window"], s["S"]), s["n_sink"]
    a = first
    while a < S:
        rows = max(16, min(1024, (1 << 28) // (s["B"] * s["H"] * min(w + 1024, S))))
        b = min(a + rows, S)
        lo = max(a - w + 1, 0)
        idx = torch.cat((torch.arange(min(ns, lo), device=DEV), torch.arange(lo, b, device=DEV)))
        row = torch.arange(a, b, device=DEV)[:, None]
        yield a, b, idx, (idx <= row) & ((idx > row - w) | (idx < ns))
        a = b


def _scores(s, a, b, idx, seen):
    """[B, Hkv, G, rows, keys] in fp32, -inf where a row does not see a key."""
    B, H, Hkv, D = (s[x] for x in ("B", "H", "Hkv", "D"))
    q = s["q"][:, a:b].float().permute(0, 2, 1, 3).reshape(B, Hkv, -1, D)
    z = (q @ s["k"][:, idx].float().permute(0, 2, 3, 1)).mul_(s["scale"])
    return z.reshape(B, Hkv, H // Hkv, b - a, -1).masked_fill_(~seen, -math.inf)


def _plain_mass(s):
    B, S, H, Hkv = (s[x] for x in ("B", "S", "H", "Hkv"))
    mass = torch.zeros(B, Hkv, S, device=DEV)
    for a, b, idx, seen in _blocks(s, S - s["n_last"]):
        p = _scores(s, a, b, idx, seen).sub_(s["lse"][:, :, a:b].reshape(B, Hkv, H // Hkv, b - a, 1)).exp_()
        mass[:, :, idx] += p.sum((2, 3))
    return mass


def _plain_step(s):
    B, S, H, Hkv, D, ns = (s[x] for x in ("B", "S", "H", "Hkv", "D", "n_sink"))
    n = s["kv_len"].long()[:, None]
    j = torch.arange(S, device=DEV)
    seen = (j < n) & ((j > n - 1 - s["window"]) | (j < ns))
    O, lse = torch.empty(B, H, D, device=DEV), torch.empty(B, H, device=DEV)
    out = torch.where(j < n[..., None], s["mass"], 0.0)
    step = max(1, (1 << 28) // (S * Hkv * D))
    for b in range(0, B, step):
        e = min(b + step, B)
        z = s["q"][b:e].float().reshape(e - b, Hkv, H // Hkv, D) @ s["k"][b:e].float().permute(0, 2, 3, 1)
        z = z.mul_(s["scale"]).masked_fill_(~seen[b:e, None, None], -math.inf)
        m = z.amax(-1, keepdim=True)
        p = torch.exp(z - torch.where(m == -math.inf, 0.0, m))
        total = p.sum(-1, keepdim=True)
        p = torch.where(total > 0, p / total, 0.0)
        O[b:e] = (p @ s["v"][b:e].float().permute(0, 2, 1, 3)).reshape(e - b, H, D)
        lse[b:e] = (m + total.log()).reshape(e - b, H)
        out[b:e] += p.sum(2)
    return O.to(torch.bfloat16), lse, out


def _plain_evict(s):
    B, S, Hkv, D, keep, cap = (s[x] for x in ("B", "S", "Hkv", "D", "keep", "cap"))
    n = s["kv_len"].long()[:, None, None]
    j = torch.arange(S, device=DEV)
    rank = torch.where((j < s["n_first"]) | (j >= n - s["n_recent"]), math.inf, s["mass"])
    rank = torch.where(j < n, rank, -math.inf)
    at = torch.sort(rank, dim=-1, descending=True, stable=True).indices[..., :keep]      # ties: the lowest positions
    at = torch.where(at < n, at, S).sort(-1).values                                      # in order, what is no key behind
    if at.shape[-1] < keep:
        at = torch.nn.functional.pad(at, (0, keep - at.shape[-1]), value=S)
    live = at < S
    kept = torch.where(live, at, -1).to(torch.int32)
    at = at.clamp(max=S - 1)
    mass = torch.zeros(B, Hkv, cap, device=DEV)
    mass[..., :keep] = torch.where(live, s["mass"].gather(-1, at), 0.0)
    out = []
    for name in ("k", "v"):
        rows = torch.take_along_dim(s[name], at.transpose(1, 2)[..., None], 1)
        t = s[name + "_out"].clone()                                                     # rows behind: as they were
        t[:, :keep] = torch.where(live.transpose(1, 2)[..., None], rows, t[:, :keep])
        out.append(t)
    return out[0], out[1], n[:, 0, 0].clamp(max=keep).to(torch.int32), mass, kept


def _plain_prefix(s):
    B, P, S, H, Hkv, D = (s[x] for x in ("B", "P", "S", "H", "Hkv", "D"))
    q = s["q"].float().reshape(B, Hkv, H // Hkv, D)
    rows = q.transpose(0, 1).reshape(Hkv, -1, D)                                         # all sequences' queries of a head
    zp = (rows @ s["k_prefix"].float().permute(1, 2, 0)).mul_(s["scale"])
    zo = (q @ s["k"].float().permute(0, 2, 3, 1)).mul_(s["scale"])
    zo.masked_fill_((torch.arange(S, device=DEV) >= s["kv_len"][:, None])[:, None, None], -math.inf)
    back = lambda t: t.reshape(Hkv, B, H // Hkv, -1).transpose(0, 1)  # noqa: E731
    m = torch.maximum(back(zp.amax(-1)), zo.amax(-1, keepdim=True))
    zp.sub_(m.transpose(0, 1).reshape(Hkv, -1, 1)).exp_()
    zo.sub_(m).exp_()
    total = back(zp.sum(-1)) + zo.sum(-1, keepdim=True)
    o = back(zp @ s["v_prefix"].float().transpose(0, 1)) + zo @ s["v"].float().permute(0, 2, 1, 3)
    return (o / total).reshape(B, H, D).to(torch.bfloat16), (m + total.log()).reshape(B, H)


# ------------------------------------------------------------------------------------------------ in 64 bits
def exact(case, seed):
    """From the definition: sequence by sequence and head by head."""
    s = prepare(case, seed)
    kind, B, S, Hkv = (s[x] for x in ("kind", "B", "S", "Hkv"))
    f64 = dict(dtype=torch.float64, device=DEV)
    if kind == "evict":
        keep, mass = s["keep"], torch.zeros(B, Hkv, s["cap"], **f64)
        k, v = s["k_out"].clone(), s["v_out"].clone()
        kept = torch.full((B, Hkv, keep), -1, dtype=torch.int32, device=DEV)
        for b, n in enumerate(_lens(s)):
            for g in range(Hkv):
                at = torch.arange(n, device=DEV)
                if n > keep:
                    lo, hi, want = s["n_first"], n - s["n_recent"], keep - s["n_first"] - s["n_recent"]
                    x = s["mass"][b, g, lo:hi]
                    border = torch.sort(x).values[len(x) - want] if want else math.inf
                    take = x > border
                    equal = torch.nonzero(x == border)[:, 0]
                    take[equal[:want - int(take.sum())]] = True
                    at = torch.cat((at[:lo], at[lo:hi][take], at[hi:]))
                m = len(at)
                kept[b, g, :m] = at
                mass[b, g, :m] = s["mass"][b, g, at].double()
                k[b, :m, g], v[b, :m, g] = s["k"][b, at, g], s["v"][b, at, g]
        return k, v, torch.tensor([min(n, keep) for n in _lens(s)], dtype=torch.int32, device=DEV), mass, kept
    H, G = s["H"], s["H"] // Hkv
    if kind == "mass":
        w, ns = s["window"], s["n_sink"]
        mass = torch.zeros(B, Hkv, S, **f64)
        for a in range(S - s["n_last"], S, 1024):
            i = torch.arange(a, min(a + 1024, S), device=DEV)[:, None]
            lo = max(0, a - w + 1)
            j = torch.cat((torch.arange(min(ns, lo), device=DEV), torch.arange(lo, int(i[-1]) + 1, device=DEV)))
            ok = (j <= i) & ((i - j < w) | (j < ns))
            for b in range(B):
                for h in range(H):
                    z = s["q"][b, i[:, 0], h].double() @ s["k"][b, j, h // G].double().T * s["scale"]
                    mass[b, h // G, j] += (torch.exp(z - s["lse"][b, h, i].double()) * ok).sum(0)
        return mass
    O = torch.zeros(B, H, s["D"], **f64)
    lse = torch.full((B, H), -math.inf, **f64)
    if kind == "prefix":
        kp, vp = s["k_prefix"].double(), s["v_prefix"].double()
    else:
        mass = s["mass"].double()
    for b, n in enumerate(_lens(s)):
        j = torch.arange(n, device=DEV)
        if kind == "step":
            j = j[(j > n - 1 - s["window"]) | (j < s["n_sink"])]
            if n == 0:
                continue
        for g in range(Hkv):
            kk, vv = s["k"][b, j, g].double(), s["v"][b, j, g].double()
            if kind == "prefix":
                kk, vv = torch.cat((kp[:, g], kk)), torch.cat((vp[:, g], vv))
            hs = slice(g * G, g * G + G)
            z = s["q"][b, hs].double() @ kk.T * s["scale"]
            lse[b, hs] = torch.logsumexp(z, -1)
            p = torch.softmax(z, -1)
            O[b, hs] = p @ vv
            if kind == "step":
                mass[b, g, j] += p.sum(0)
    return (O, lse, mass) if kind == "step" else (O, lse)
