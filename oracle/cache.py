"""The target's cache operators in fp64: head norms and rotation, attention
under a window with sinks, eviction by weight.

Plain restatements of the definitions for the tests; one sequence at a time,
caches as contiguous rows (pages are the tests' business).
"""
from __future__ import annotations

import numpy as np


def norm_rotate(x, gain, eps, pos, inv_freq, interleaved):
    """x [n, heads, dh], pos [n] -> rows after the norm (gain None: none) and the rotation."""
    y = np.array(x, dtype=np.float64)
    if gain is not None:
        y = y / np.sqrt((y * y).mean(-1, keepdims=True) + eps) * np.asarray(gain, np.float64)
    for i, f in enumerate(inv_freq):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + len(inv_freq))
        ang = np.asarray(pos, np.float64)[:, None] * f
        c, s = np.cos(ang), np.sin(ang)
        ya, yb = y[..., a].copy(), y[..., b].copy()
        y[..., a], y[..., b] = ya * c - yb * s, yb * c + ya * s
    return y


def visible(pq, pk, window, sinks):
    """[n, L] mask: query positions pq [n], row positions pk [L]."""
    pq, pk = np.asarray(pq, np.int64)[:, None], np.asarray(pk, np.int64)[None]
    see = pk <= pq
    if window:
        see &= (pq - pk < window) | (pk < sinks)
    return see


def attention(q, k, v, pq, pk, scale, window=0, sinks=0, there=None):
    """q [n, Hq, dh], k, v [L, Hkv, dh], pk [L, Hkv], there [L] (rows that exist).

    Returns out [n, Hq, dh], lse [n, Hq], the weight [L, Hkv] the rows get, sum p |v|
    [n, Hq, dh] and the largest sum |q k| scale of a visible pair (for error bounds).
    """
    q, k, v = (np.asarray(t, np.float64) for t in (q, k, v))
    n, hq, dh = q.shape
    L, hkv = k.shape[0], k.shape[1]
    out, mag = np.zeros((n, hq, dh)), np.zeros((n, hq, dh))
    lse, weight, big = np.full((n, hq), -np.inf), np.zeros((L, hkv)), 0.0
    for h in range(hq):
        g = h // (hq // hkv)
        see = visible(pq, pk[:, g], window, sinks)
        if there is not None:
            see &= np.asarray(there)[None]
        rows = see.any(0)
        if not rows.any():
            continue
        kk, vv, see = k[rows, g], v[rows, g], see[:, rows]
        s = np.where(see, q[:, h] @ kk.T * scale, -np.inf)
        big = max(big, float((np.abs(q[:, h]) @ np.abs(kk).T * scale).max()))
        some = see.any(1)
        top = np.where(some, s.max(1, initial=-np.inf), 0.0)
        e = np.exp(s - top[:, None])
        tot = e.sum(1)
        p = e / np.where(some, tot, 1.0)[:, None]
        out[:, h], mag[:, h] = p @ vv, p @ np.abs(vv)
        lse[some, h] = top[some] + np.log(tot[some])
        weight[rows, g] += p.sum(0)
    return out, lse, weight, mag, big


def evict(weight, pos, next_pos, budget, sinks, recent):
    """Moves (to, from) of one head's rows: weight, pos [L]; none when L <= budget."""
    L = len(pos)
    if L <= budget:
        return []
    w = np.where(np.asarray(weight, np.float64) > 0, weight, 0.0)
    safe = [r for r in range(L) if pos[r] < sinks or pos[r] >= next_pos - recent]
    rest = sorted(set(range(L)) - set(safe), key=lambda r: (-w[r], r))
    kept = set((safe + rest)[:budget])
    holes = [r for r in range(budget) if r not in kept]
    movers = [r for r in range(budget, L) if r in kept]
    return list(zip(holes, movers))
