"""Causal attention of packed prompts in float64 (test infrastructure only)."""
from __future__ import annotations

import numpy as np


def prompt_attention(q: np.ndarray, k: np.ndarray, v: np.ndarray, q_lens, k_lens, scale: float):
    """q [total_q, Hq, D], k / v [total_k, Hkv, D] float64.  Returns (out, sum_j p_j |v_j|) per element;
    rows without keys are zero."""
    hq, group = q.shape[1], q.shape[1] // k.shape[1]
    out, size = np.zeros(q.shape), np.zeros(q.shape)
    q0 = k0 = 0
    for lq, lk in zip(q_lens, k_lens):
        for r in range(lq):
            n = r + lk - lq + 1
            if n <= 0:
                continue
            for h in range(hq):
                g = h // group
                s = scale * (k[k0:k0 + n, g] @ q[q0 + r, h])
                p = np.exp(s - s.max())
                p /= p.sum()
                out[q0 + r, h] = p @ v[k0:k0 + n, g]
                size[q0 + r, h] = p @ np.abs(v[k0:k0 + n, g])
        q0, k0 = q0 + lq, k0 + lk
    return out, size
