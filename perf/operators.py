"""The sliding-window attention with sinks and the 8-bit attention checkpoints, as they are measured.

Five kinds of case:
  fwd      causal attention in which a query sees the last `window` tokens and the first `n_sink` ones
  bwd      its gradients from the saved output and log-sum-exp
  decode   its form for a single new token of each sequence, over a cache with a length for each sequence
  ckpt     q, k, v and O of one attention layer saved in 8 bits, and restored
  ckptbwd  q, k, v and O saved in 8 bits, and the gradients computed from what was saved

With `own` False, `run` computes them with elementary torch operations in 32 bits; with `own` True it makes the
library's calls.  Shapes: q, O, dO [B, S, H, D], k, v [B, S, Hkv, D] in bf16, lse [B, H, S] in fp32.
"""
import math

import torch

own = False

DEV = "cuda"
GROUP = 32          # elements of the head dimension that share one exponent in a checkpoint
CASE_MAX = 32768 * (4096 + 256) * 32    # score elements of the largest listed case's band


# ------------------------------------------------------------------------------------------------ cases
def listed():
    return [
        # a short prompt of a small model: the call's latency counts
        dict(name="fwd short", kind="fwd", B=1, S=129, H=4, Hkv=4, D=64, window=32, n_sink=1),
        # a training batch of ragged length, grouped heads, the window's edge inside tiles
        dict(name="fwd ragged batch", kind="fwd", B=2, S=5003, H=16, Hkv=2, D=128, window=1000, n_sink=7),
        # one long training sequence: 32 heads over 8 key/value heads
        dict(name="fwd 32K", kind="fwd", B=1, S=32768, H=32, Hkv=8, D=128, window=4096, n_sink=4),
        # gradients of a short odd batch at the small head dim
        dict(name="bwd short", kind="bwd", B=2, S=777, H=8, Hkv=4, D=64, window=200, n_sink=8),
        # gradients of one long training sequence
        dict(name="bwd 32K", kind="bwd", B=1, S=32768, H=32, Hkv=8, D=128, window=4096, n_sink=4),
        # a quarter of the heads of a 128K sequence (heads split over steps), a wide sink
        dict(name="bwd 128K", kind="bwd", B=1, S=131072, H=8, Hkv=2, D=128, window=2048, n_sink=64),
        # a single user's next token
        dict(name="decode one", kind="decode", B=1, S=2048, H=32, Hkv=8, D=128, window=1024, n_sink=4, lo=1501, hi=1501),
        # a server's batch of next tokens over long caches of different lengths, some shorter than the window
        dict(name="decode batch", kind="decode", B=32, S=16384, H=32, Hkv=8, D=128, window=8192, n_sink=4, lo=1, hi=16384),
        # a small layer's checkpoint, odd length
        dict(name="ckpt small", kind="ckpt", B=1, S=501, H=8, Hkv=8, D=64),
        # the checkpoint of one layer of a 32K sequence
        dict(name="ckpt 32K", kind="ckpt", B=1, S=32768, H=32, Hkv=8, D=128),
        # a training step's backward from the checkpoint, short and causal over the whole sequence
        dict(name="ckptbwd causal", kind="ckptbwd", B=1, S=1500, H=8, Hkv=2, D=128, window=1500, n_sink=0),
        # the same for a windowed layer of a longer sequence
        dict(name="ckptbwd 16K", kind="ckptbwd", B=1, S=16384, H=32, Hkv=8, D=128, window=2048, n_sink=4),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    kind = rng.choice(["fwd", "bwd", "decode", "ckpt", "ckptbwd"])
    D = rng.choice([64, 128])
    Hkv = rng.choice([1, 2, 4, 8])
    H = Hkv * rng.choice([1, 2, 3, 4, 8])
    B = rng.choice([1, 1, 2, 3])
    if kind == "decode":
        B, S = _log(rng, 1, 48), _log(rng, 1, 16384)
        hi = rng.randint(1, S)
        return dict(kind=kind, B=B, S=S, H=H, Hkv=Hkv, D=D, window=_log(rng, 1, 16384), n_sink=rng.choice([0, 1, 4, 17, 128]),
                    lo=rng.randint(0, hi), hi=hi)
    if kind == "ckpt":
        return dict(kind=kind, B=B, S=_log(rng, 1, 32768 // B), H=H, Hkv=Hkv, D=D)
    # a query that sees itself alone has gradients of zero, which only rounding fills: not for the backward
    least = 1 if kind == "fwd" else 2
    S, window, n_sink = _log(rng, least, 131072), _log(rng, least, 8192), rng.choice([0, 1, 4, 33, 128])
    while B * H * (S + 256) * (min(window, S) + 256) > CASE_MAX // 2:
        S = S * 3 // 4
    return dict(kind=kind, B=B, S=S, H=H, Hkv=Hkv, D=D, window=window, n_sink=n_sink)


def _lens(case):
    n = case["B"]
    return [case["lo"] + (case["hi"] - case["lo"]) * b // max(n - 1, 1) for b in range(n)]


def _pairs(case):
    """Visible (query, key) pairs of one head of one sequence."""
    S, w, ns = case["S"], case["window"], case["n_sink"]
    w = min(w, S)
    band = w * (w + 1) // 2 + (S - w) * w
    n = min(ns, S - w)                       # sink j is outside the window of queries i >= j + w
    return band + n * (S - w) - n * (n - 1) // 2


def work(case):
    B, S, H, Hkv, D, kind = (case[x] for x in ("B", "S", "H", "Hkv", "D", "kind"))
    q, kv = B * S * H * D, B * S * Hkv * D
    if kind == "decode":
        keys = sum(min(n, case["window"]) + min(case["n_sink"], max(n - case["window"], 0)) for n in _lens(case))
        return {"bytes": 4 * keys * Hkv * D + 4 * B * H * D + 4 * B * H + 4 * B, "flops": 4 * D * H * keys}
    held = (2 * q + 2 * kv) * (1 + 1 / GROUP)
    if kind == "ckpt":                       # read in bf16, held in 8 bits, read back, written in bf16
        return {"bytes": 2 * (2 * q + 2 * kv) * 2 + 2 * held, "flops": 4 * (2 * q + 2 * kv)}
    pairs, lse = B * H * _pairs(case), 4 * B * H * S
    if kind == "fwd":
        return {"bytes": 2 * (2 * q + 2 * kv) + lse, "flops": 4 * D * pairs}
    read = 2 * (2 * q + 2 * kv) + (2 * held if kind == "ckptbwd" else 0)
    return {"bytes": read + 2 * q + lse + 2 * (q + 2 * kv), "flops": 10 * D * pairs}


# ------------------------------------------------------------------------------------------------ inputs
def prepare(case, seed):
    """Unit-normal activations; the sinks' keys lie along the direction that all queries share (they draw a few
    times an ordinary token's weight) and their values are small, as trained sinks are."""
    B, S, H, Hkv, D, kind = (case[x] for x in ("B", "S", "H", "Hkv", "D", "kind"))
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    rnd = lambda *shape: torch.randn(shape, generator=gen, device=DEV)  # noqa: E731
    ns = min(case.get("n_sink", 0), S)
    u = rnd(Hkv, D)
    q = rnd(B, 1 if kind == "decode" else S, H, D) + 0.25 * u.repeat_interleave(H // Hkv, 0)
    k, v = rnd(B, S, Hkv, D), rnd(B, S, Hkv, D)
    k[:, :ns] = 0.3 * k[:, :ns] + 1.5 * u
    v[:, :ns] *= 0.1
    q, k, v = (t.to(torch.bfloat16) for t in (q, k, v))
    state = dict(case, q=q, k=k, v=v, scale=D ** -0.5)
    if kind == "decode":
        state["q"] = q[:, 0]
        state["kv_len"] = torch.tensor(_lens(case), dtype=torch.int32, device=DEV)
    elif kind == "ckpt":
        state["O"] = rnd(B, S, H, D).to(torch.bfloat16)
    elif kind in ("bwd", "ckptbwd"):
        state["O"], state["lse"] = _plain_fwd(q, k, v, case["window"], case["n_sink"], state["scale"])
        state["dO"] = rnd(B, S, H, D).to(torch.bfloat16)
    return state


# ------------------------------------------------------------------------------------------------ one pass
def run(state):
    s = state
    if own:
        return _own(s)
    if s["kind"] == "fwd":
        return _plain_fwd(s["q"], s["k"], s["v"], s["window"], s["n_sink"], s["scale"])
    if s["kind"] == "bwd":
        return _plain_bwd(s["q"], s["k"], s["v"], s["O"], s["lse"], s["dO"], s["window"], s["n_sink"], s["scale"])
    if s["kind"] == "decode":
        return _plain_decode(s["q"], s["k"], s["v"], s["kv_len"], s["window"], s["n_sink"], s["scale"])
    held = tuple(_held_in_8(s[x].float()) for x in ("q", "k", "v", "O"))
    if s["kind"] == "ckpt":
        return tuple(t.to(torch.bfloat16) for t in held)
    return _plain_bwd(*held, s["lse"], s["dO"], s["window"], s["n_sink"], s["scale"])


def _own(s):
    from long_context_causal_gb300 import dfa
    if s["kind"] == "fwd":
        return dfa.dfa_attn_fwd_sink(s["q"], s["k"], s["v"], s["window"], s["n_sink"], scale=s["scale"])
    if s["kind"] == "bwd":
        return dfa.dfa_attn_bwd_sink(s["q"], s["k"], s["v"], s["O"], s["lse"], s["dO"], s["window"], s["n_sink"],
                                     scale=s["scale"])
    if s["kind"] == "decode":
        return dfa.dfa_attn_decode_sink(s["q"], s["k"], s["v"], s["kv_len"], s["window"], s["n_sink"], scale=s["scale"])
    ckpt = dfa.dfa_ckpt8_save(s["q"], s["k"], s["v"], s["O"])
    if s["kind"] == "ckpt":
        return dfa.dfa_ckpt8_restore(ckpt, s["B"], s["H"], s["Hkv"], s["S"], s["D"])
    return dfa.dfa_attn_bwd_ckpt8(ckpt, s["lse"], s["dO"], s["Hkv"], s["window"], s["n_sink"], scale=s["scale"])


# ------------------------------------------------------------------------------------------------ plain forms
def _held_in_8(x):
    """What 8 bits hold of x: groups of 32 along the last axis share an exponent e = floor(log2 max|x|) - 6, an
    element is the integer nearest to x / 2^e (ties to even, at most 127 in magnitude)."""
    g = x.reshape(*x.shape[:-1], -1, GROUP)
    amax = g.abs().amax(-1, keepdim=True)
    e = (torch.frexp(amax).exponent - 7).clamp(min=-120)
    up, down = (((127 + n) << 23).view(torch.float32) for n in (e, -e))     # 2^e and 2^-e, from their bits
    return (torch.round(g * down).clamp(-127, 127) * up).reshape(x.shape)


def _bands(q, k, v, window, n_sink, scale):
    """Queries in blocks of rows, each block's keys and values as one band, and the sinks apart.  Returns
    (q blocks [B, g, n, G*blk, D], k and v bands [B, g, n, width, D], sink k and v [B, g, 1, ns, D], scores of
    the band and of the sinks (masked with -inf), the band's first key position, (blk, width, G))."""
    B, S, H, D = q.shape
    Hkv = k.shape[2]
    G, w = H // Hkv, min(window, S)
    blk = min(256, S)
    n = -(-S // blk)
    width, pad = blk + w - 1, n * blk - S
    qb = _blocks(q, blk, Hkv)
    kb, vb = (torch.nn.functional.pad(t.float().permute(0, 2, 1, 3), (0, 0, w - 1, pad)).unfold(2, width, blk).transpose(3, 4).contiguous()
              for t in (k, v))
    ks, vs = (t[:, :n_sink].float().permute(0, 2, 1, 3)[:, :, None] for t in (k, v))
    row = torch.arange(n, device=q.device)[:, None] * blk + torch.arange(blk, device=q.device)   # [n, blk]
    row = row.repeat(1, G)[..., None]                                                           # [n, G*blk, 1]
    key = torch.arange(n, device=q.device)[:, None, None] * blk - (w - 1) + torch.arange(width, device=q.device)
    sink = torch.arange(ks.shape[3], device=q.device)
    sb = (qb @ kb.transpose(3, 4)).mul_(scale)
    sb.masked_fill_((key > row) | (key <= row - w) | (key < 0) | (key >= S), -math.inf)
    ss = (qb @ ks.transpose(3, 4)).mul_(scale)
    ss.masked_fill_(sink > row - w, -math.inf)          # a sink inside the window is in the band already
    return qb, kb, vb, ks, vs, sb, ss, (blk, width, G, n)


def _blocks(x, blk, Hkv):
    """[B, S, H, D] -> fp32 [B, Hkv, n, G*blk, D], rows past the end zero."""
    B, S, H, D = x.shape
    n = -(-S // blk)
    x = torch.nn.functional.pad(x.float(), (0, 0, 0, 0, 0, n * blk - S)).reshape(B, n, blk, Hkv, H // Hkv, D)
    return x.permute(0, 3, 1, 4, 2, 5).reshape(B, Hkv, n, -1, D)


def _unblock(x, S, G):
    """The inverse of _blocks."""
    B, Hkv, n, r, D = x.shape
    return x.reshape(B, Hkv, n, G, r // G, D).permute(0, 2, 4, 1, 3, 5).reshape(B, n * (r // G), Hkv * G, D)[:, :S]


def _plain_fwd(q, k, v, window, n_sink, scale):
    S = q.shape[1]
    qb, kb, vb, ks, vs, sb, ss, (blk, width, G, n) = _bands(q, k, v, window, n_sink, scale)
    m = torch.cat((sb.amax(-1, keepdim=True), ss), -1).amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, 0.0, m)             # rows past the end
    sb.sub_(m).exp_()
    ss.sub_(m).exp_()
    total = sb.sum(-1, keepdim=True) + ss.sum(-1, keepdim=True)
    o = (sb @ vb + ss @ vs) / total
    lse = _unblock(m + total.log(), S, G)[..., 0].transpose(1, 2)
    return _unblock(o, S, G).to(torch.bfloat16).contiguous(), lse.contiguous()


def _plain_bwd(q, k, v, O, lse, dO, window, n_sink, scale):
    B, S, H, D = q.shape
    Hkv = k.shape[2]
    qb, kb, vb, ks, vs, pb, ps, (blk, width, G, n) = _bands(q, k, v, window, n_sink, scale)
    ns, w = ks.shape[3], min(window, S)
    lb = _blocks(lse.transpose(1, 2)[..., None], blk, Hkv)
    db, ob = _blocks(dO, blk, Hkv), _blocks(O, blk, Hkv)
    delta = (db * ob).sum(-1, keepdim=True)
    pb.sub_(lb).exp_()
    ps.sub_(lb).exp_()
    key = (torch.arange(n, device=q.device)[:, None] * blk + torch.arange(width, device=q.device)).reshape(-1)

    def by_key(band, sinks):                            # the bands' shares of each key, and the sinks'
        out = torch.zeros(B, Hkv, n * blk + w - 1, D, device=q.device)
        out.index_add_(2, key, band.reshape(B, Hkv, -1, D))
        out = out[:, :, w - 1:w - 1 + S].clone()
        out[:, :, :ns] += sinks.sum(2)
        return out.transpose(1, 2).to(torch.bfloat16).contiguous()

    dv = by_key(pb.transpose(3, 4) @ db, ps.transpose(3, 4) @ db)
    pb.mul_((db @ vb.transpose(3, 4)).sub_(delta))
    ps.mul_((db @ vs.transpose(3, 4)).sub_(delta))
    dk = by_key((pb.transpose(3, 4) @ qb).mul_(scale), (ps.transpose(3, 4) @ qb).mul_(scale))
    dq = _unblock((pb @ kb + ps @ ks).mul_(scale), S, G).to(torch.bfloat16).contiguous()
    return dq, dk, dv


def _plain_decode(q, k, v, kv_len, window, n_sink, scale):
    B, S, Hkv, D = k.shape
    H, w = q.shape[1], min(window, S)
    n = kv_len.long()[:, None]
    sink = torch.arange(min(n_sink, S), device=q.device).expand(B, -1)
    near = n - w + torch.arange(w, device=q.device)
    at = torch.cat((sink, near), 1)
    seen = torch.cat((sink < n - w, near >= 0), 1)      # a sink inside the window is there already
    at = at.clamp(0, S - 1)
    kk, vv = (torch.take_along_dim(t, at[:, :, None, None], 1).float().permute(0, 2, 1, 3) for t in (k, v))
    s = (q.float().reshape(B, Hkv, H // Hkv, D) @ kk.transpose(2, 3)).mul_(scale)
    s.masked_fill_(~seen[:, None, None], -math.inf)
    m = s.amax(-1, keepdim=True)
    p = torch.exp(s - torch.where(m == -math.inf, 0.0, m))
    total = p.sum(-1, keepdim=True)
    o = torch.where(total > 0, (p @ vv) / total, 0.0)
    return o.reshape(B, H, D).to(torch.bfloat16), (m + total.log()).reshape(B, H)


# ------------------------------------------------------------------------------------------------ in 64 bits
def exact(case, seed):
    """From the definition, tile of rows by tile of rows and head by head."""
    s = prepare(case, seed)
    kind, S, w, ns, G = s["kind"], s["S"], s.get("window"), s.get("n_sink"), s["H"] // s["Hkv"]
    f64 = dict(dtype=torch.float64, device=DEV)

    def eight(x):
        out = torch.empty_like(x)
        for a in range(0, x.shape[-1], GROUP):
            g = x[..., a:a + GROUP]
            big = g.abs().amax(-1, keepdim=True)
            mant = torch.frexp(big).mantissa
            step = torch.where(big > 0, big / (mant * 128), 1.0)        # big = mant 2^n: 2^(n - 7), exactly
            out[..., a:a + GROUP] = torch.round(g / step).clamp(-127, 127) * step
        return out

    def tiles():
        step = max(256, min(2048, (1 << 27) // (min(w, S) + 2048)))
        for b in range(s["B"]):
            for g in range(s["Hkv"]):
                for a in range(0, S, step):
                    i = torch.arange(a, min(a + step, S), device=DEV)
                    lo = max(0, a - w + 1)
                    j = torch.cat((torch.arange(min(ns, lo), device=DEV), torch.arange(lo, int(i[-1]) + 1, device=DEV)))
                    ok = (j[None] <= i[:, None]) & ((j[None] > i[:, None] - w) | (j[None] < ns))
                    for h in range(g * G, g * G + G):
                        yield b, g, h, i, j, ok

    if kind == "decode":
        O = torch.zeros(s["B"], s["H"], s["D"], **f64)
        lse = torch.full((s["B"], s["H"]), -math.inf, **f64)
        for b, n in enumerate(_lens(s)):
            j = torch.arange(n, device=DEV)
            j = j[(j > n - 1 - w) | (j < ns)]
            kk, vv, qq = s["k"][b, j].double(), s["v"][b, j].double(), s["q"][b].double()
            for h in range(s["H"] if n else 0):
                z = kk[:, h // G] @ qq[h] * s["scale"]
                lse[b, h] = torch.logsumexp(z, 0)
                O[b, h] = torch.softmax(z, 0) @ vv[:, h // G]
        return O, lse
    q, k, v = (s[x].double() for x in ("q", "k", "v"))
    if kind == "fwd":
        O, lse = torch.empty_like(q), torch.empty(s["B"], s["H"], S, **f64)
        for b, g, h, i, j, ok in tiles():
            z = (q[b, i, h] @ k[b, j, g].T * s["scale"]).masked_fill(~ok, -math.inf)
            lse[b, h, i] = torch.logsumexp(z, -1)
            O[b, i, h] = torch.softmax(z, -1) @ v[b, j, g]
        return O, lse
    O = s["O"].double()
    if kind != "bwd":
        q, k, v, O = eight(q), eight(k), eight(v), eight(O)
    if kind == "ckpt":
        return q, k, v, O
    dO, lse = s["dO"].double(), s["lse"].double()
    dq, dk, dv = torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)
    for b, g, h, i, j, ok in tiles():
        d = dO[b, i, h]
        p = torch.exp(q[b, i, h] @ k[b, j, g].T * s["scale"] - lse[b, h, i, None]) * ok
        ds = p * (d @ v[b, j, g].T - (d * O[b, i, h]).sum(-1, keepdim=True)) * s["scale"]
        dq[b, i, h] = ds @ k[b, j, g]
        dk[b, j, g] += ds.T @ q[b, i, h]
        dv[b, j, g] += p.T @ d
    return dq, dk, dv
