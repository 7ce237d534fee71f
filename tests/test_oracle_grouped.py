"""Pins of the block-128, grouped and routing oracle: restatements from the definitions."""

from fractions import Fraction

import numpy as np
import pytest

import oracle


def e4m3_codes():
    codes = np.array([c for c in range(128) if c != 0x7F])
    return codes, [Fraction(float(v)) for v in oracle.e4m3_value(codes)]


def nearest_code(q: Fraction) -> int:
    """The E4M3 code nearest to a rational, by search over all values; ties to the even code."""
    codes, values = e4m3_codes()
    mag = min(abs(q), Fraction(448))
    best = min(range(len(codes)), key=lambda i: (abs(values[i] - mag), codes[i] & 1))
    return int(codes[best]) | (0x80 if q < 0 else 0)


def test_codes_are_the_nearest_of_the_exact_quotient():
    # every pair of 8-bit significands: where ties are, and how near the others come
    closest = Fraction(1)
    for ma in range(128, 256, 9):
        x = np.arange(128, 256) * 2.0 ** -3
        block = np.zeros(256)
        block[:128], block[128] = np.where(x > ma, 0.0, x), 0.0
        block[127] = ma  # amax
        q, s = oracle.quantize_b128(block)
        assert s[0] == np.float32(ma) / np.float32(448) and s[1] == 0
        for i in range(0, 127, 5):
            exact = Fraction(float(block[i])) * 448 / ma
            assert q[i] == nearest_code(exact), (ma, i)
            for c in range(16, 32):  # ties lie half way between neighbours of 4 significant bits
                e = 0
                while Fraction(2 * c + 1, 2) * Fraction(2) ** e > 2 * exact and exact > 0:
                    e -= 1
                tie = Fraction(2 * c + 1, 2) * Fraction(2) ** e
                if exact > 0 and tie != exact:
                    closest = min(closest, abs(exact - tie) / tie)
    assert closest > Fraction(1, 2 ** 14)


def test_special_blocks():
    x = np.zeros((5, 128))
    x[1, 3] = -0.0
    x[2, 7] = np.inf
    x[3, 9] = np.nan
    x[4, 0], x[4, 1] = 448.0, -1.0
    q, s = oracle.quantize_b128(x)
    assert s[0] == 0 and s[1] == 0 and np.isnan(s[2]) and np.isnan(s[3]) and s[4] == 1
    assert (q[2] == 0x7F).all() and (q[3] == 0x7F).all()
    assert q[4, 0] == 0x7E and q[4, 1] == 0xB8
    assert (q[0] == 0).all() and q[1, 3] == 0x80


@pytest.mark.parametrize("N,K", [(128, 128), (130, 272), (1, 16)])
def test_weight_blocks_restated(N, K):
    w = np.random.default_rng(N + K).standard_normal((2, N, K)).astype(np.float32).astype(np.float64)
    q, s = oracle.quantize_weights_b128(w)
    assert s.shape == (2, -(-N // 128), -(-K // 128))
    for b in range(2):
        for i in range(s.shape[1]):
            for j in range(s.shape[2]):
                blk = w[b, 128 * i:128 * i + 128, 128 * j:128 * j + 128]
                assert s[b, i, j] == np.float32(np.abs(blk).max()) / np.float32(448)
    # E4M3 keeps 2^-4 of a value, and 2^-10 of the block's step below its normal range
    err = np.abs(oracle.dequantize_weights_b128(q, s) - w)
    wide = np.repeat(np.repeat(s, 128, -1)[..., :K], 128, -2)[..., :N, :]
    assert (err <= np.maximum(np.abs(w) * 2.0 ** -4, wide * 2.0 ** -10) * (1 + 1e-6)).all()


def test_grouped_restated():
    rng = np.random.default_rng(0)
    x, w, b = rng.integers(-4, 5, (9, 6)), rng.integers(-4, 5, (4, 3, 6)), rng.integers(-4, 5, (4, 3))
    off = [0, 2, 2, 7, 8]
    out = oracle.grouped(x.astype(float), w.astype(float), off, b.astype(float))
    of_row = [0, 0, 2, 2, 2, 2, 2, 3]
    for r, e in enumerate(of_row):
        for n in range(3):
            assert out[r, n] == sum(int(x[r, k]) * int(w[e, n, k]) for k in range(6)) + b[e, n]
    assert np.isnan(out[8]).all()


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
def test_route_restated(scoring):
    rng = np.random.default_rng(5)
    z = rng.integers(-3, 4, (40, 7)).astype(float)  # many ties
    z[3] = -np.inf
    z[5, 1:] = np.nan
    r = oracle.route(z, 3, scoring)
    assert (r["ids"][3] == -1).all() and (r["positions"][3] == -1).all() and (r["weights"][3] == 0).all()
    assert list(r["ids"][5]) == [0, -1, -1]
    for t in range(40):
        got = [e for e in r["ids"][t] if e >= 0]
        left = dict(enumerate(np.where(np.isnan(z[t]), -np.inf, z[t])))
        for e in got:  # one largest after the other, the first of equals
            assert e == max(left, key=lambda i: (left[i], -i))
            del left[e]
        for j, e in enumerate(got):
            p = r["positions"][t, j]
            assert r["offsets"][e] <= p < r["offsets"][e + 1] and r["rows"][p] == t
            with np.errstate(invalid="ignore"):
                ex = np.where(np.isnan(z[t]), 0, np.exp(np.where(np.isnan(z[t]), 0, z[t])))
            want = ex[e] / ex.sum() if scoring == "softmax" else ex[e] / (1 + ex[e])
            assert abs(r["weights"][t, j] - want) < 1e-12
    n = r["offsets"][-1]
    assert (r["rows"][n:] == -1).all() and n == (r["ids"] >= 0).sum()
    for e in range(7):
        assert list(r["rows"][r["offsets"][e]:r["offsets"][e + 1]]) == sorted(r["rows"][r["offsets"][e]:r["offsets"][e + 1]])


def test_combine_restated():
    y = np.arange(12.0).reshape(4, 3)
    out = oracle.combine(y, np.array([[1, 3], [-1, 0], [4, -1]]), np.array([[2.0, 0.5], [9.0, 1.0], [1.0, 1.0]]), np.ones((3, 3)))
    assert np.array_equal(out, np.stack([2 * y[1] + 0.5 * y[3] + 1, y[0] + 1, np.ones(3)]))


def test_a_planted_mistake_is_seen():
    """The oracle's neighbours are other numbers: a scale of the wrong block, a tie away from even."""
    x = np.zeros(128)
    x[0], x[1] = 64.0, 17.0 / 7.0  # 448 x / amax = 17 exactly: between 16 and 18, 16 is even
    q, _ = oracle.quantize_b128(np.float64(x) * 7)
    assert oracle.e4m3_value(q[1]) == 16.0
    assert oracle.e4m3_value(q[1]) != 18.0
