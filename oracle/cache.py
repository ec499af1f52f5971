"""CPU oracle for the calls on a key/value cache -- TEST INFRASTRUCTURE ONLY.

Rotary positions, attention of drafted tokens over a cache, and eviction, each
written out from its definition in float64 with NumPy. Shares no code with the
CUDA library.
"""
from __future__ import annotations

import math

import numpy as np


def rotate(X, pos, inv_freq, interleaved=False, transpose=False, factor=1.0):
    """X [B,H,T,d] at positions pos [B,T]: pairs turned by pos * inv_freq."""
    X = np.array(X, dtype=np.float64)
    n = len(inv_freq)
    a = np.asarray(pos, dtype=np.float64)[:, None, :, None] * np.asarray(inv_freq, dtype=np.float64)
    c, s = factor * np.cos(a), factor * np.sin(a) * (-1.0 if transpose else 1.0)
    i, j = (slice(0, 2 * n, 2), slice(1, 2 * n, 2)) if interleaved else (slice(0, n), slice(n, 2 * n))
    x, y = X[..., i].copy(), X[..., j].copy()
    X[..., i], X[..., j] = x * c - y * s, x * s + y * c
    return X


def ancestors(parents, T):
    """sees[t, j]: drafted token t sees drafted token j (itself or an ancestor)."""
    sees = np.zeros((T, T), dtype=bool)
    for t in range(T):
        a = t
        while a >= 0:
            sees[t, a] = True
            a = int(parents[a]) if parents is not None else a - 1
    return sees


def tree_attn(Q, K, V, length, parents, n, scale):
    """One sequence: Q [Hq,T,d], K, V [Hkv,cap,d], n drafted tokens. Returns
    O [Hq,n,d], lse [Hq,n], p_slots [Hkv,length+n], abs_v [Hq,n,d] (sum p |v|)
    and abs_s (the largest scale * sum |q||k|), the last two for error bounds."""
    Hq, Hkv = Q.shape[0], K.shape[0]
    G = Hq // Hkv
    d = Q.shape[-1]
    O, A = np.zeros((Hq, n, d)), np.zeros((Hq, n, d))
    lse = np.full((Hq, n), -math.inf)
    W = np.zeros((Hkv, length + n))
    abs_s = 0.0
    sees = ancestors(parents, n)
    for hq in range(Hq):
        k, v = K[hq // G, : length + n], V[hq // G, : length + n]
        for t in range(n):
            seen = np.concatenate([np.ones(length, dtype=bool), sees[t]])
            s = scale * (k[seen] @ Q[hq, t])
            abs_s = max(abs_s, scale * float((np.abs(k[seen]) @ np.abs(Q[hq, t])).max()))
            top = s.max()
            e = np.exp(s - top)
            p = e / e.sum()
            lse[hq, t] = top + math.log(e.sum())
            O[hq, t], A[hq, t] = p @ v[seen], p @ np.abs(v[seen])
            W[hq // G, np.flatnonzero(seen)] += p
    return O, lse, W, A, abs_s


def evict_rows(weight, pos, length, n_draft, accept, keep, sinks, recent, next_pos):
    """One (sequence, kv head): the source slot of each slot below m, by the rule."""
    cand = list(range(length)) + [length + j for j in range(n_draft) if accept is None or (int(accept) >> j) & 1]
    m = min(keep, len(cand))

    def rank(i):
        held = pos[i] < sinks or (next_pos is not None and pos[i] >= int(next_pos) - recent)
        w = float(weight[i])
        return (not held, (1, 0.0) if math.isnan(w) else (0, -w), i) if not held else (False, (0, 0.0), i)

    kept = set(sorted(cand, key=rank)[:m])
    come = iter(sorted(i for i in kept if i >= m))
    return [i if i in kept else next(come) for i in range(m)]
