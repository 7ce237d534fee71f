"""The 4-bit oracle's NVFP4 rule where 6 g is zero or leaves the normal fp32 range (CPU)."""

import numpy as np
import pytest

import oracle


@pytest.mark.parametrize("g", [0.0, 1e-45, 1e-40, 1.0, 6e37])
def test_a_zero_block_has_the_scale_zero(g):
    codes, s = oracle.quantize4(np.zeros((1, 32)), "nvfp4", g)
    assert not codes.any() and not s.any()
    assert not oracle.dequantize4(codes, s, "nvfp4", g).any()


def test_g_zero_gives_the_value_zero():
    x = np.zeros((1, 32))
    x[0, 17] = 3.0
    codes, s = oracle.quantize4(x, "nvfp4", 0.0)
    assert s.tolist() == [[0, 0x7E]] and not codes.any()  # 3 / 2^-149 saturates, s g = 0 gives zero codes
    assert not oracle.dequantize4(codes, s, "nvfp4", 0.0).any()


def test_subnormal_g_by_hand():
    g = float(np.float32(2.0 ** -135))  # 6 g = 1.5 * 2^-133, whose inverse fp32 does not hold
    x = np.zeros((1, 32))
    x[0, 2], x[0, 18] = 6 * g, 12 * g
    codes, s = oracle.quantize4(x, "nvfp4", g)
    assert s.tolist() == [[0x38, 0x40]]  # 1 and 2
    assert not codes.any()               # 1 / g overflows: s g is below what can be inverted
