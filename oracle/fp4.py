"""The 4-bit cache format in float64: codes, scales, tiles.

Test infrastructure only (see ``oracle/__init__``).

* e2m1: 1 sign, 2 exponent bits (bias 1), 1 mantissa bit; no infinities, no NaN.
* 16 elements of a row share one e4m3 scale; the value of an element is code * scale * head scale.
* Quantising: u = x / head scale (the quotient rounded to fp32); s = the e4m3 value nearest to
  max|u| / 6 (quotient rounded to fp32; ties to the even code), within 2^-9 .. 448; the code is the
  e2m1 value nearest to u / s, ties to the even code, saturating.  A NaN makes s the NaN code.
* A tile is 16 rows: [16][D / 2] code bytes (even element in the low nibble), [16][D / 16] scales.
"""
from __future__ import annotations

import numpy as np

from .formats import e4m3_table


def e2m1_value(code: int) -> float:
    sign, exp, man = code >> 3, (code >> 1) & 3, code & 1
    mag = 0.5 * man if exp == 0 else (1.0 + 0.5 * man) * 2.0 ** (exp - 1)
    return -mag if sign else mag


E2M1 = np.array([e2m1_value(c) for c in range(16)])


def _nearest_even(x: np.ndarray, grid: np.ndarray) -> np.ndarray:
    """Index of the grid value nearest to each x (grid ascending from 0, x within it); ties to even."""
    d = np.abs(x[..., None] - grid)
    best = d.min(-1, keepdims=True)
    tied = d == best
    even = tied & (np.arange(len(grid)) % 2 == 0)
    return np.where(even.any(-1), even.argmax(-1), tied.argmax(-1))


def quantise(x: np.ndarray, head_scale=None):
    """x float64 [..., heads, D] -> (codes uint8 [..., D] in 0..15, scale codes uint8 [..., D / 16])."""
    x32 = np.asarray(x, dtype=np.float64).astype(np.float32)
    with np.errstate(all="ignore"):
        if head_scale is not None:
            x32 = x32 / np.asarray(head_scale, dtype=np.float32)[:, None]
        u = x32.reshape(x32.shape[:-1] + (x32.shape[-1] // 16, 16))
        mx = np.max(np.abs(np.where(np.isnan(u), np.float32(0), u)), -1)
        want = np.clip((mx / np.float32(6)).astype(np.float64), 2.0 ** -9, 448.0)
    grid = e4m3_table()[:0x7F]
    sc = _nearest_even(want, grid).astype(np.uint8)
    s = grid[sc][..., None]
    with np.errstate(all="ignore"):
        mag = np.minimum(np.abs(u.astype(np.float64)) / s, 6.0)
    nan = np.isnan(u)
    code = _nearest_even(np.where(nan, 0.0, mag), E2M1[:8]) + 8 * np.signbit(u)
    sc = np.where(nan.any(-1), 0x7F, sc).astype(np.uint8)
    return code.astype(np.uint8).reshape(x32.shape), sc


def values(codes: np.ndarray, scale_codes: np.ndarray) -> np.ndarray:
    """float64 code * scale, [..., D]."""
    v = E2M1[codes].reshape(codes.shape[:-1] + (codes.shape[-1] // 16, 16)) * e4m3_table()[scale_codes][..., None]
    return v.reshape(codes.shape)


def pack(codes: np.ndarray, scale_codes: np.ndarray) -> np.ndarray:
    """[NB, heads, B, D] codes and [NB, heads, B, D / 16] scales -> pool uint8 [NB, heads, B / 16, 9 D]."""
    nb, h, b, d = codes.shape
    by = (codes[..., 0::2] | (codes[..., 1::2] << 4)).reshape(nb, h, b // 16, 8 * d)
    return np.concatenate([by, scale_codes.reshape(nb, h, b // 16, d)], -1)


def unpack(pool: np.ndarray):
    """The inverse of pack."""
    nb, h, tiles, nbytes = pool.shape
    d = nbytes // 9
    by = pool[..., : 8 * d].reshape(nb, h, tiles * 16, d // 2)
    codes = np.stack([by & 15, by >> 4], -1).reshape(nb, h, tiles * 16, d)
    return codes, pool[..., 8 * d:].reshape(nb, h, tiles * 16, d // 16)
