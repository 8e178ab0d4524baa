"""fp64 reference of windowed attention with sinks, its gradients, its
single-token form and the 8-bit checkpoint -- TEST INFRASTRUCTURE ONLY.

Dense numpy arithmetic from the definitions: a query at position i sees key j
iff j <= i and (j > i - window or j < n_sink), and
  s = scale <q, k>,  lse = ln sum exp(s),  P = exp(s - lse),  O = P v,
  Delta = <dO, O>,  dS = P (dO v^T - Delta),
  dQ = scale dS K,  dK = scale dS^T Q,  dV = P^T dO  (summed over a GQA group).
Beside each result it returns the sum of the magnitudes of the result's terms,
which is what a rounding of the terms by a relative u moves it by at most, u
times over: the tests' tolerances are built from them.

Layouts: q, O, dO [B, S, H, D], k, v [B, S, H_kv, D], lse [B, H, S].
"""
from __future__ import annotations

import numpy as np

GROUP = 32


def visible(S: int, window: int, n_sink: int) -> np.ndarray:
    i, j = np.arange(S)[:, None], np.arange(S)[None]
    return (j <= i) & ((j > i - window) | (j < n_sink))


def _scores(q, k, h, scale):
    return scale * (q[:, h] @ k[:, h // (q.shape[1] // k.shape[1])].T)


def attn_fwd(q, k, v, window, n_sink, scale=None):
    """O, lse and sum_j P_ij |v_j|."""
    q, k, v = (np.asarray(t, dtype=np.float64) for t in (q, k, v))
    B, S, H, D = q.shape
    G = H // k.shape[2]
    scale = D ** -0.5 if scale is None else scale
    see = visible(S, window, n_sink)
    O, size, lse = np.zeros_like(q), np.zeros_like(q), np.zeros((B, H, S))
    for b in range(B):
        for h in range(H):
            s = np.where(see, _scores(q[b], k[b], h, scale), -np.inf)
            m = s.max(1, keepdims=True)
            p = np.exp(s - m)
            total = p.sum(1, keepdims=True)
            lse[b, h] = (m + np.log(total))[:, 0]
            O[b, :, h] = p / total @ v[b, :, h // G]
            size[b, :, h] = p / total @ np.abs(v[b, :, h // G])
    return O, lse, size


def attn_bwd(q, k, v, O, lse, dO, window, n_sink, scale=None, most=np.inf):
    """Gradients from the given O and lse: {"dQ": (value, terms, cancel, floor), ...}.
    `terms` sums |dS| |k|, |dS| |q| or P |dO|; `cancel` sums P (|dO| |v|^T +
    |dO| |O|) |k| (or |q|): what dO v^T - Delta is the difference of (0 for dV);
    `floor` is `cancel` with P = 1 on every visible pair: what an absolute error
    of P moves the result by.  `most`: what P counts as at most in dS (with the
    forward's lse it is 1 at most)."""
    q, k, v, O, lse, dO = (np.asarray(t, dtype=np.float64) for t in (q, k, v, O, lse, dO))
    B, S, H, D = q.shape
    G = H // k.shape[2]
    scale = D ** -0.5 if scale is None else scale
    see = visible(S, window, n_sink)
    out = {n: tuple(np.zeros_like(t) for _ in range(4)) for n, t in (("dQ", q), ("dK", k), ("dV", v))}
    for b in range(B):
        for h in range(H):
            g = h // G
            qh, kh, vh, oh, dh = q[b, :, h], k[b, :, g], v[b, :, g], O[b, :, h], dO[b, :, h]
            p = np.where(see, np.exp(_scores(q[b], k[b], h, scale) - lse[b, h][:, None]), 0.0)
            pv, p = p, np.minimum(p, most)
            ds = p * (dh @ vh.T - (dh * oh).sum(1, keepdims=True)) * scale
            f = see * (np.abs(dh) @ np.abs(vh).T + (np.abs(dh) * np.abs(oh)).sum(1, keepdims=True)) * scale
            for z, w in enumerate((ds, np.abs(ds), p * f, f)):
                kk, qq = (kh, qh) if z == 0 else (np.abs(kh), np.abs(qh))
                out["dQ"][z][b, :, h] += w @ kk
                out["dK"][z][b, :, g] += w.T @ qq
            out["dV"][0][b, :, g] += pv.T @ dh
            out["dV"][1][b, :, g] += pv.T @ np.abs(dh)
    return out


def decode(q, k, v, kv_len, window, n_sink, scale=None):
    """One query per sequence, at position kv_len[b] - 1: O [B, H, D], lse [B, H]
    and sum_j P_j |v_j|.  Rows of k and v that are not visible are never used."""
    q = np.asarray(q, dtype=np.float64)
    B, H, D = q.shape
    G = H // k.shape[2]
    scale = D ** -0.5 if scale is None else scale
    O, size, lse = np.zeros_like(q), np.zeros_like(q), np.full((B, H), -np.inf)
    for b in range(B):
        n = int(kv_len[b])
        j = np.arange(n)
        j = j[(j > n - 1 - window) | (j < n_sink)]
        if j.size == 0:
            continue
        kk, vv = np.asarray(k[b][j], dtype=np.float64), np.asarray(v[b][j], dtype=np.float64)
        for h in range(H):
            s = scale * (kk[:, h // G] @ q[b, h])
            m = s.max()
            p = np.exp(s - m)
            lse[b, h] = m + np.log(p.sum())
            O[b, h] = p / p.sum() @ vv[:, h // G]
            size[b, h] = p / p.sum() @ np.abs(vv[:, h // G])
    return O, lse, size


def ckpt8(x):
    """What the 8-bit checkpoint holds of x [..., D]."""
    x = np.asarray(x, dtype=np.float64)
    g = x.reshape(*x.shape[:-1], -1, GROUP)
    big = np.abs(g).max(-1, keepdims=True)
    bad = ~np.isfinite(big)
    e = np.maximum(np.frexp(np.where(bad, 1.0, big))[1] - 1 - 6, -120)
    m = np.clip(np.rint(np.ldexp(np.where(bad, 0.0, g), -e)), -127, 127)
    return np.where(bad, np.nan, np.ldexp(m, e)).reshape(x.shape)
