"""Attention of new rows over a cache and eviction by attention weight, in float64 (test infrastructure only)."""
from __future__ import annotations

import numpy as np


def chunk_attention(q, k, v, start: int, scale: float):
    """One sequence: q [n, Hq, D] at positions start .. start + n - 1, k and v [start + n, Hkv, D], float64.
    Returns (out, lse [n, Hq], sum_j p_j |v_j|); a row sees keys 0 .. start + r and nothing else."""
    n, hq, _ = q.shape
    group = hq // k.shape[1]
    out, size, lse = np.zeros(q.shape), np.zeros(q.shape), np.zeros((n, hq))
    with np.errstate(all="ignore"):
        for h in range(hq):
            kh, vh = k[:, h // group], v[:, h // group]
            for r in range(n):
                m = start + r + 1
                s = scale * (kh[:m] @ q[r, h])
                top = s.max()
                e = np.exp(s - top)
                lse[r, h] = top + np.log(e.sum())
                p = e / e.sum()
                out[r, h] = p @ vh[:m]
                size[r, h] = p @ np.abs(vh[:m])
    return out, lse, size


def chunk_weights(q, lse, k, start: int, scale: float):
    """w [Hkv, start + n]: each key's exp(scale q . k - lse), summed over the rows that see it and its query heads."""
    n, hq, _ = q.shape
    hkv = k.shape[1]
    w = np.zeros((hkv, start + n))
    for h in range(hq):
        for r in range(n):
            m = start + r + 1
            w[h // (hq // hkv), :m] += np.exp(scale * (k[:m, h // (hq // hkv)] @ q[r, h]) - lse[r, h])
    return w


def select(weights, length: int, keep: int, first: int, recent: int):
    """Positions one head keeps of its weights [>= length], ascending."""
    n = min(keep, length)
    order = []
    order += [(0, -j) for j in range(length - recent, length) if j >= 0]            # the newest, from the end
    taken = set(-j for _, j in order)
    order += [(1, j) for j in range(min(first, length)) if j not in taken]
    taken |= set(j for c, j in order if c == 1)
    rest = [j for j in range(length) if j not in taken]
    key = lambda j: (-weights[j] if not np.isnan(weights[j]) else np.inf, np.isnan(weights[j]), j)  # noqa: E731
    ranked = [-j if c == 0 else j for c, j in sorted(order)] + sorted(rest, key=key)
    return sorted(ranked[:n])


def compact(cache, kept, keep, src_tables, dst_tables, block: int):
    """A copy of rows [blocks, Hkv, block, ...] after the move; every source is read before any row is written."""
    out = cache.copy()
    for i, n in enumerate(keep):
        for h in range(cache.shape[1]):
            for j in range(n):
                p = kept[i][h][j]
                if p >= 0:
                    out[dst_tables[i][j // block], h, j % block] = cache[src_tables[i][p // block], h, p % block]
    return out
