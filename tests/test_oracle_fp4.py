"""The 4-bit oracle against hand-worked values and exhaustive searches (CPU)."""

import numpy as np
import pytest

import oracle


def test_e2m1_rounds_to_nearest_even_code_and_saturates():
    x = np.array([0.0, 0.25, 0.26, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 5.01, 7.9, 1e30])
    want = np.array([0.0, 0.0, 0.5, 1.0, 1.0, 2.0, 2.0, 4.0, 4.0, 6.0, 6.0, 6.0])
    assert np.array_equal(oracle.e2m1_value(oracle.e2m1_encode(x)), want)
    assert np.array_equal(oracle.e2m1_value(oracle.e2m1_encode(-x)), -want)
    assert oracle.e2m1_encode(np.array([-0.0]))[0] == 8


def test_e2m1_codes_round_trip_and_are_nearest():
    codes = np.arange(16, dtype=np.uint8)
    assert np.array_equal(oracle.e2m1_encode(oracle.e2m1_value(codes)), codes)
    x = np.linspace(-6.5, 6.5, 4001)
    got = oracle.e2m1_value(oracle.e2m1_encode(x))
    best = np.min(np.abs(x[:, None] - oracle.e2m1_value(codes)[None, :]), axis=1)
    assert np.array_equal(np.abs(x - got), best)


def test_pack_puts_the_even_element_low():
    q = oracle.pack(np.array([[1, 2, 15, 8]], dtype=np.uint8))
    assert q.tolist() == [[0x21, 0x8F]]
    assert oracle.unpack(q).tolist() == [[1, 2, 15, 8]]


def test_mxfp4_scale_is_the_power_of_two_under_amax_over_four():
    x = np.zeros((1, 64))
    x[0, 0], x[0, 1], x[0, 40] = 7.0, -1.0, 0.75  # e = 0 and e = -1 - 2
    codes, s = oracle.quantize4(x, "mxfp4")
    assert s.tolist() == [[127, 124]]
    v = oracle.dequantize4(codes, s, "mxfp4")
    assert v[0, 0] == 6.0 and v[0, 1] == -1.0 and v[0, 40] == 0.75


def test_nvfp4_scale_and_value():
    x = np.zeros((1, 32))
    x[0, 3], x[0, 20] = 12.0, -0.5
    codes, s = oracle.quantize4(x, "nvfp4", g=1.0)
    assert s.tolist() == [[0x40, 0x1B]]  # 2.0, and 0.5 / 6 = 0.0833 -> 1.375 * 2^-4
    v = oracle.dequantize4(codes, s, "nvfp4", 1.0)
    assert v[0, 3] == 12.0
    assert abs(v[0, 20] + 0.5) <= 0.5 * 2 ** -4  # the E4M3 scale's half step


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
def test_blocks_with_nan_inf_or_zero(fmt):
    n = oracle.fp4_oracle.BLOCKS[fmt]
    x = np.ones((1, 4 * n))
    x[0, 1], x[0, n + 2], x[0, 2 * n:3 * n] = np.nan, np.inf, 0.0
    codes, s = oracle.quantize4(x, fmt)
    assert s[0, :2].tolist() == ([0xFF] * 2 if fmt == "mxfp4" else [0x7F] * 2)
    assert not codes[0, :3 * n].any() and s[0, 2] == 0
    assert np.allclose(oracle.dequantize4(codes[:, 3 * n:], s[:, 3:], fmt), 1.0, rtol=0.07)


def test_norm_and_activation_by_hand():
    t, y = oracle.rmsnorm([[3.0, 4.0]], [1.0, 2.0], [[0.0, 0.0]], eps=0.0)
    assert np.allclose(y, [[3 / np.sqrt(12.5), 8 / np.sqrt(12.5)]])
    assert oracle.silu_mul([0.0, 1.0], [5.0, 2.0]).tolist() == [0.0, 2.0 / (1 + np.exp(-1.0))]
