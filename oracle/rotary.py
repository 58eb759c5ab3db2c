"""Rotation by position and per-head RMS norm in float64 (test infrastructure only)."""
from __future__ import annotations

import math

import numpy as np


def frequencies(rotary_dim: int, base: float, scaling: str = "none", factor: float = 1.0,
                original_context: float = 0.0, alpha: float = 1.0, beta: float = 32.0) -> np.ndarray:
    """f_i in radians per position."""
    if scaling == "ntk":
        base = base * factor ** (rotary_dim / (rotary_dim - 2))
    out = []
    for i in range(rotary_dim // 2):
        f = base ** (-2.0 * i / rotary_dim)
        if scaling == "linear":
            f = f / factor
        if scaling == "parts":
            r = original_context * f / (2 * math.pi)         # turns over the original context
            keep = min(max((r - alpha) / (beta - alpha), 0.0), 1.0)
            f = keep * f + (1 - keep) * f / factor
        out.append(f)
    return np.array(out)


def rms_norm(x: np.ndarray, weight, eps: float) -> np.ndarray:
    return x if weight is None else x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * weight


def rotate(x: np.ndarray, positions: np.ndarray, freq: np.ndarray, layout: str, magnitude: float = 1.0):
    """x [tokens, heads, D]; returns the rotated rows and, per element, |a| + |b| of its pair (for error bounds)."""
    half = len(freq)
    ang = positions.astype(np.float64)[:, None] * freq
    cos, sin = magnitude * np.cos(ang)[:, None], magnitude * np.sin(ang)[:, None]
    ia = np.arange(half) if layout == "half" else 2 * np.arange(half)
    ib = ia + half if layout == "half" else ia + 1
    y, size = x.copy(), np.abs(x)
    a, b = x[..., ia], x[..., ib]
    y[..., ia], y[..., ib] = a * cos - b * sin, b * cos + a * sin
    size[..., ia] = size[..., ib] = np.abs(a) + np.abs(b)
    return y, size * magnitude if magnitude > 1 else size
