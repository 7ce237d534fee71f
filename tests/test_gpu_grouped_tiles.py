"""Block-128 and grouped products on every kernel and tile width that is not split along K, CTA pairs above
all: exact sums with bias, ragged rows, columns and K, and nothing written around the output.  Which shape
goes where is held by test_grouped_plan_cpu.py."""

import numpy as np
import pytest
import torch

import oracle
from _grouped import (assert_product, bf16_round, codes, f64, fake, offsets_of, pack, product_bound, to_bf16, to_dev,
                      weights)
from _grouped_shapes import BATCHED, DENSE, GROUPED, GROUPED_RAGGED_K
from _helpers import device
from mxfp8_block_scaled_02_gb300 import ops

pytestmark = pytest.mark.gpu
BAND = 4096
WHOLE = oracle.e4m3_encode(np.arange(-2.0, 3.0))  # codes of -2 .. 2


def whole_numbers(rng, *shape):
    """(values, codes): half of them 0, the others -2 .. 2."""
    v = np.where(rng.random(shape) < 0.5, rng.integers(-2, 3, shape), 0)
    return v.astype(np.float64), WHOLE[v + 2]


def powers(rng, *shape):
    return np.exp2(rng.integers(-2, 3, shape))


def exact_rows(rng, fmt, *shape):
    """(values, codes, scales) of rows [..., R, K].  With exact_weights all products are multiples of
    2^-4 of at most 2^6, so that fp32 sums of up to 2^14 of them are exact in any order."""
    v, q = whole_numbers(rng, *shape)
    K = shape[-1]
    if fmt == "fp8_128":
        s = powers(rng, *shape[:-1], -(-K // 128))
        return v * np.repeat(s, 128, -1)[..., :K], q, s.astype(np.float32)
    s = powers(rng, *shape[:-1], K // 32)
    return v * np.repeat(s, 32, -1), q, (127 + np.log2(s)).astype(np.uint8)


def exact_weights(rng, fmt, *shape):
    if fmt == "mxfp8":
        return exact_rows(rng, fmt, *shape)
    N, K = shape[-2:]
    v, q = whole_numbers(rng, *shape)
    s = powers(rng, *shape[:-2], -(-N // 128), -(-K // 128))
    return v * np.repeat(np.repeat(s, 128, -1)[..., :K], 128, -2)[..., :N, :], q, s.astype(np.float32)


def banded(n, dev):
    return torch.full((2 * BAND + n,), 0xA5, dtype=torch.uint8, device=dev)


def assert_bands(t):
    assert (t[:BAND] == 0xA5).all() and (t[-BAND:] == 0xA5).all()


def check_dense(lead, N, K):
    dev = device()
    rng = np.random.default_rng(lead[-1] * 7 + N * 3 + K)
    x, xq, xs = exact_rows(rng, "fp8_128", *lead, K)
    w, wq, ws = exact_weights(rng, "fp8_128", *lead[:-1], N, K)
    ref = x @ w.swapaxes(-1, -2)
    bias = rng.integers(-8, 9, N).astype(np.float64)
    pw = ops.process_weights_fp8_128(to_dev(wq, dev), to_dev(ws, dev))
    xd, sd = to_dev(xq, dev), to_dev(xs, dev)
    buf = banded(2 * ref.size, dev)
    out = buf[BAND:-BAND].view(torch.bfloat16).view(ref.shape)
    ops.linear_fp8_128(xd, pw, to_bf16(bias, dev), sd, out=out)
    ops.check()
    assert_bands(buf)
    assert np.array_equal(f64(out), bf16_round(ref + bias))
    assert np.array_equal(f64(ops.linear_fp8_128(xd, pw, x_scale=sd)), bf16_round(ref))


@pytest.mark.parametrize("M,N,K", [shape for shape, _ in DENSE])
def test_dense(M, N, K):
    check_dense((M,), N, K)


@pytest.mark.parametrize("B,M,N,K", [shape for shape, _ in BATCHED])
def test_batched(B, M, N, K):
    check_dense((B, M), N, K)


@pytest.mark.parametrize("fmt,case", [(fmt, c) for c in GROUPED for fmt in ("mxfp8", "fp8_128")] +
                         [("fp8_128", c) for c in GROUPED_RAGGED_K])
def test_grouped(fmt, case):
    counts, N, K, _ = case
    dev = device()
    R, E = sum(counts), len(counts)
    rng = np.random.default_rng(R + N + K)
    x, xq, xs = exact_rows(rng, fmt, R, K)
    w, wq, ws = exact_weights(rng, fmt, E, N, K)
    bias = rng.integers(-8, 9, (E, N)).astype(np.float64)
    off = offsets_of(counts)
    pw, xd, sd, od = pack(ops, wq, ws, fmt, dev), to_dev(xq, dev), to_dev(xs, dev), to_dev(off, dev)
    need = ops.grouped_workspace_size(pw.fmt, E, R, N, K, True)
    buf, room = banded(2 * R * N, dev), banded(need, dev)
    out = buf[BAND:-BAND].view(torch.bfloat16).view(R, N)
    ops.grouped_linear(xd, pw, od, sd, bias=to_bf16(bias, dev), out=out, workspace=room[BAND:-BAND])
    ops.check()
    assert_bands(buf)
    assert_bands(room)
    assert np.array_equal(f64(out), bf16_round(oracle.grouped(x, w, off, bias)))
    assert np.array_equal(f64(ops.grouped_linear(xd, pw, od, sd)), bf16_round(oracle.grouped(x, w, off)))
    # the first and last rows of no group: left as they were, the others' results unchanged
    lo, hi = counts[0] // 2, R - counts[-1] // 2
    od = to_dev(np.clip(off, lo, hi).astype(np.int32), dev)
    kept = torch.full((R, N), 7.0, dtype=torch.bfloat16, device=dev)
    ops.grouped_linear(xd, pw, od, sd, bias=to_bf16(bias, dev), out=kept)
    ops.check()
    assert torch.equal(kept[lo:hi], out[lo:hi]) and (kept[:lo] == 7).all() and (kept[hi:] == 7).all()


@pytest.mark.parametrize("M,N,K", [(515, 4104, 400), (2049, 1032, 272)])
def test_bf16_rows_dense(M, N, K):
    dev = device()
    rng = np.random.default_rng(M)
    q, s, w = weights(rng, "fp8_128", N, K)
    x = bf16_round(rng.standard_normal((M, K)) * np.where(rng.random((M, K)) < 1e-3, 100.0, 1.0))
    bias = bf16_round(rng.standard_normal(N))
    pw = ops.process_weights_fp8_128(to_dev(q, dev), to_dev(s, dev))
    room = banded(ops.workspace_size_fp8_128(1, M, N, K, False), dev)
    out = ops.linear_fp8_128(to_bf16(x, dev), pw, to_bf16(bias, dev), workspace=room[BAND:-BAND])
    ops.check()
    assert_bands(room)
    xf = fake(x, "fp8_128")
    ref = xf @ w.T + bias
    assert_product(out, ref, product_bound(xf, w, ref))
    xq, xs = codes(x, "fp8_128")
    assert torch.equal(out, ops.linear_fp8_128(to_dev(xq, dev), pw, to_bf16(bias, dev), to_dev(xs, dev)))


@pytest.mark.parametrize("fmt", ["mxfp8", "fp8_128"])
def test_bf16_rows_grouped(fmt):
    dev = device()
    counts, N, K, _ = GROUPED[2]
    R, E = sum(counts), len(counts)
    rng = np.random.default_rng(R)
    q, s, w = weights(rng, fmt, E, N, K)
    x = bf16_round(rng.standard_normal((R, K)) * np.where(rng.random((R, K)) < 1e-3, 100.0, 1.0))
    off, bias = offsets_of(counts), bf16_round(rng.standard_normal((E, N)))
    pw = pack(ops, q, s, fmt, dev)
    out = ops.grouped_linear(to_bf16(x, dev), pw, to_dev(off, dev), bias=to_bf16(bias, dev))
    ops.check()
    xf = fake(x, fmt)
    ref = oracle.grouped(xf, w, off, bias)
    bound = np.concatenate([product_bound(xf[off[e]:off[e + 1]], w[e], ref[off[e]:off[e + 1]]) for e in range(E)])
    assert_product(out, ref, bound)
    xq, xs = codes(x, fmt)
    assert torch.equal(out, ops.grouped_linear(to_dev(xq, dev), pw, to_dev(off, dev), to_dev(xs, dev), bias=to_bf16(bias, dev)))
