"""fp64 reference of the calls over a long cache: attention weights gathered per
key, the keys that stay, attention behind a shared prefix -- TEST INFRASTRUCTURE ONLY.

Plain numpy from the definitions:
  mass_j   = sum over a group's heads h and the last n_last queries i that see j
             of exp(scale <q_ih, k_j> - lse_ih), queries and keys as in oracle.sink;
  kept     = the first n_first, the last n_recent and the heaviest others, the
             lower position where masses are equal, NaN below every number;
  prefix   : softmax attention of one query over P shared keys and n own ones.

Layouts: q [B, S, H, D] (one token: [B, H, D]), k, v [B, S, H_kv, D], prefixes
[P, H_kv, D], lse [B, H, S], mass [B, H_kv, S].
"""
from __future__ import annotations

import numpy as np

from oracle import sink


def mass(q, k, lse, window, n_sink, n_last, scale=None):
    q, k, lse = (np.asarray(t, dtype=np.float64) for t in (q, k, lse))
    B, S, H, D = q.shape
    Hkv = k.shape[2]
    scale = D ** -0.5 if scale is None else scale
    see = sink.visible(S, window, n_sink)[S - n_last:]
    out = np.zeros((B, Hkv, S))
    for b in range(B):
        for h in range(H):
            s = scale * (q[b, S - n_last:, h] @ k[b, :, h * Hkv // H].T)
            with np.errstate(invalid="ignore", over="ignore"):
                out[b, h * Hkv // H] += np.where(see, np.exp(s - lse[b, h, S - n_last:, None]), 0.0).sum(0)
    return out


def step_mass(q, k, kv_len, window, n_sink, scale=None):
    """The weights that one query per sequence gives its keys, [B, H_kv, S_max]."""
    q = np.asarray(q, dtype=np.float64)
    B, H, D = q.shape
    S, Hkv = k.shape[1:3]
    scale = D ** -0.5 if scale is None else scale
    out = np.zeros((B, Hkv, S))
    for b in range(B):
        n = int(kv_len[b])
        j = np.arange(n)
        j = j[(j > n - 1 - window) | (j < n_sink)]
        for h in range(H if j.size else 0):
            g = h * Hkv // H
            s = scale * (np.asarray(k[b][j, g], dtype=np.float64) @ q[b, h])
            p = np.exp(s - s.max())
            out[b, g, j] += p / p.sum()
    return out


def kept(mass_row, n, keep, n_first, n_recent):
    """The positions that stay of a row's n keys, rising."""
    if n <= keep:
        return np.arange(n)
    x = np.array(mass_row[:n], dtype=np.float64)
    free = np.arange(n_first, n - n_recent)
    # heaviest first; numbers before NaN, equal ones by position
    order = sorted(free, key=lambda j: (np.isnan(x[j]), -x[j] if not np.isnan(x[j]) else 0.0, j))
    return np.sort(np.concatenate((np.arange(n_first), np.arange(n - n_recent, n),
                                   np.array(order[:keep - n_first - n_recent], dtype=np.int64)))).astype(np.int64)


def decode_prefix(q, kp, vp, k, v, kv_len, scale=None):
    """O, lse and sum_j P_j |v_j| of one query per sequence over the prefix and its own rows."""
    q, kp, vp = (np.asarray(t, dtype=np.float64) for t in (q, kp, vp))
    B, H, D = q.shape
    Hkv = k.shape[2]
    scale = D ** -0.5 if scale is None else scale
    O, size, lse = np.zeros_like(q), np.zeros_like(q), np.full((B, H), -np.inf)
    for b in range(B):
        n = int(kv_len[b])
        kk = np.concatenate((kp, np.asarray(k[b][:n], dtype=np.float64)))
        vv = np.concatenate((vp, np.asarray(v[b][:n], dtype=np.float64)))
        for h in range(H if len(kk) else 0):
            s = scale * (kk[:, h * Hkv // H] @ q[b, h])
            p = np.exp(s - s.max())
            lse[b, h] = s.max() + np.log(p.sum())
            O[b, h] = p / p.sum() @ vv[:, h * Hkv // H]
            size[b, h] = p / p.sum() @ np.abs(vv[:, h * Hkv // H])
    return O, lse, size
