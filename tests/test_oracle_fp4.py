"""Pins of the 4-bit format's oracle, the rotary oracle and the prompt oracle (CPU)."""
import math

import numpy as np
import pytest
import torch

from oracle import fp4, prompt, rotary


def test_e2m1_values():
    assert list(fp4.E2M1[:8]) == [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]
    assert list(fp4.E2M1[8:]) == [-0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0]


def test_ties_go_to_the_even_code():
    # amax 6 gives scale 1, so the elements are the quotients themselves
    x = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0, -0.25, -0.75, -1.25, -1.75, -2.5, -3.5, -5.0, 0.0])
    codes, sc = fp4.quantise(x[None])
    assert fp4.e4m3_table()[sc].item() == 1.0
    assert list(fp4.values(codes, sc)[0]) == [0, 1, 1, 2, 2, 4, 4, 6, 0, -1, -1, -2, -2, -4, -4, 0]


def test_quantising_quantised_values_changes_nothing():
    rng = np.random.default_rng(3)
    codes = rng.integers(0, 16, (50, 3, 64)).astype(np.uint8)
    codes[..., 0::16] = 7                                   # every group holds a 6
    sc = rng.integers(1, 0x7F, (50, 3, 4)).astype(np.uint8)
    c2, s2 = fp4.quantise(fp4.values(codes, sc))
    assert np.array_equal(s2, sc) and np.array_equal(fp4.values(c2, s2), fp4.values(codes, sc))


def test_small_large_nan_and_zero_groups():
    x = np.zeros((1, 4 * 16))
    x[0, 3] = 0.004                                         # below 6 * 2^-9: the smallest scale
    x[0, 16] = 1e30                                         # saturates: 6 * 448
    x[0, 33] = np.nan
    codes, sc = fp4.quantise(x)
    v = fp4.values(codes, sc)[0]
    assert list(sc[0]) == [1, 0x7E, 0x7F, 1]
    assert v[3] == 2.0 * 2.0 ** -9 and v[16] == 2688.0
    assert np.isnan(v[32:48]).all() and (v[48:] == 0).all()


def test_error_is_at_most_half_a_step():
    rng = np.random.default_rng(5)
    x = rng.standard_normal((200, 2, 128)).astype(np.float32).astype(np.float64)
    hs = np.array([0.7, 1.9], dtype=np.float32)
    codes, sc = fp4.quantise(x, hs)
    v = fp4.values(codes, sc) * hs.astype(np.float64)[:, None]
    s = np.repeat(fp4.e4m3_table()[sc], 16, -1) * hs.astype(np.float64)[:, None]
    # steps are 0.5 s below 2 s, s below 4 s, 2 s above; past 6 s (a scale rounded down by up to 1/16) saturation
    step = np.where(np.abs(x) <= 2 * s, 0.5, np.where(np.abs(x) <= 4 * s, 1.0, 2.0)) * s
    assert (np.abs(v - x) <= np.maximum(step / 2, np.abs(x) - 6 * s) * (1 + 1e-6)).all()


def test_pack_round_trip():
    rng = np.random.default_rng(7)
    codes = rng.integers(0, 16, (3, 2, 32, 64)).astype(np.uint8)
    sc = rng.integers(0, 256, (3, 2, 32, 4)).astype(np.uint8)
    pool = fp4.pack(codes, sc)
    assert pool.shape == (3, 2, 2, 576)
    # the documented bytes: row 17, element 5 is the high nibble of byte 2 of tile row 1
    assert pool[1, 1, 1, 1 * 32 + 2] >> 4 == codes[1, 1, 17, 5]
    assert pool[1, 1, 1, 16 * 32 + 1 * 4 + 3] == sc[1, 1, 17, 3]
    c2, s2 = fp4.unpack(pool)
    assert np.array_equal(c2, codes) and np.array_equal(s2, sc)


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_rotation_is_a_complex_product_and_keeps_relative_positions(layout):
    rng = np.random.default_rng(11)
    f = rotary.frequencies(32, 10000.0)
    x = rng.standard_normal((2, 3, 48))
    y, _ = rotary.rotate(x, np.array([7, 19]), f, layout)
    assert np.array_equal(y[..., 32:], x[..., 32:])
    assert np.allclose((y ** 2).sum(-1), (x ** 2).sum(-1))
    # q at 7 . k at 19 equals q at 107 . k at 119
    z, _ = rotary.rotate(x, np.array([107, 119]), f, layout)
    assert np.allclose((y[0] * y[1]).sum(-1), (z[0] * z[1]).sum(-1))
    # position 1, pair 0 turns by one radian
    e = np.zeros((1, 1, 48))
    e[..., 0] = 1.0
    w, _ = rotary.rotate(e, np.array([1]), f, layout)
    assert math.isclose(w[0, 0, 0], math.cos(1)) and math.isclose(w[0, 0, 16 if layout == "half" else 1], math.sin(1))


def test_frequency_scaling_ends():
    f = rotary.frequencies(64, 10000.0)
    assert np.allclose(rotary.frequencies(64, 10000.0, "linear", 4.0), f / 4)
    ntk = rotary.frequencies(64, 10000.0, "ntk", 4.0)
    assert ntk[0] == 1.0 and math.isclose(ntk[-1], f[-1] / 4)      # the slowest pair is interpolated fully
    parts = rotary.frequencies(64, 10000.0, "parts", 4.0, 4096.0, 1.0, 32.0)
    r = 4096.0 * f / (2 * math.pi)
    assert np.allclose(parts[r >= 32], f[r >= 32]) and np.allclose(parts[r <= 1], f[r <= 1] / 4)
    assert (np.diff(parts) < 0).all()


def test_prompt_oracle_is_bottom_right_causal_attention():
    rng = np.random.default_rng(13)
    lq, lk = [5, 0, 3, 4], [9, 2, 3, 2]
    q, k, v = (rng.standard_normal((sum(n), h, 16)) for n, h in ((lq, 4), (lk, 2), (lk, 2)))
    out, _ = prompt.prompt_attention(q, k, v, lq, lk, 0.25)
    q0 = k0 = 0
    for a, b in zip(lq, lk):
        mask = torch.ones(a, b, dtype=torch.bool).tril(b - a)
        qq = torch.from_numpy(q[q0:q0 + a]).transpose(0, 1)
        kk, vv = (torch.from_numpy(t[k0:k0 + b]).transpose(0, 1).repeat_interleave(2, 0) for t in (k, v))
        ref = torch.nn.functional.scaled_dot_product_attention(qq, kk, vv, attn_mask=mask, scale=0.25).transpose(0, 1)
        ref = torch.nan_to_num(ref).numpy() if a else ref.numpy()
        assert np.allclose(out[q0:q0 + a], ref)
        q0, k0 = q0 + a, k0 + b
