"""Products grouped by expert (MXFP8 and block-128 FP8) against the fp64 oracle."""

import numpy as np
import pytest
import torch

import oracle
from _grouped import (assert_product, bf16_round, codes, f64, fake, offsets_of, pack, product_bound, to_bf16, to_dev,
                      weights)
from _helpers import device
from mxfp8_block_scaled_02_gb300 import ops

pytestmark = pytest.mark.gpu
FMTS = ["mxfp8", "fp8_128"]

# (rows of each expert, N, K): none, one, tile edges of every kernel, very uneven; K a multiple of 128
CASES = [
    ([1], 8, 128),
    ([0, 3, 0, 0, 1, 16, 0], 136, 256),
    ([17, 0, 31, 32, 33, 1], 264, 384),
    ([64, 65, 1, 0, 96], 128, 640),
    ([128, 0, 129, 3], 392, 256),
    ([0, 700, 0, 256, 257, 5], 520, 384),
    ([1030, 12], 264, 512),
    ([1] * 40 + [0] * 23 + [9], 256, 256),
    ([0, 0, 0], 128, 128),
    ([2] * 300, 8, 128),
]


def exact_case(rng, fmt, counts, N, K):
    """Whole-number codes and power-of-two scales: exact in fp32."""
    R, E = int(sum(counts)), len(counts)
    xv = rng.integers(-2, 3, (R, K)) * (rng.random((R, K)) < 0.5)
    wv = rng.integers(-2, 3, (E, N, K)) * (rng.random((E, N, K)) < 0.5)
    xq, wq = oracle.e4m3_encode(xv.astype(np.float64)), oracle.e4m3_encode(wv.astype(np.float64))
    if fmt == "fp8_128":
        xs = np.exp2(rng.integers(-2, 3, (R, K // 128))).astype(np.float32)
        ws = np.exp2(rng.integers(-2, 3, (E, -(-N // 128), K // 128))).astype(np.float32)
        return xq, xs, wq, ws, oracle.dequantize_b128(xq, xs), oracle.dequantize_weights_b128(wq, ws)
    xs = (127 + rng.integers(-2, 3, (R, K // 32))).astype(np.uint8)
    ws = (127 + rng.integers(-2, 3, (E, N, K // 32))).astype(np.uint8)
    return xq, xs, wq, ws, oracle.dequantize(xq, xs), oracle.dequantize(wq, ws)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("case", range(len(CASES)))
def test_exact_sums(fmt, case):
    counts, N, K = CASES[case]
    dev = device()
    rng = np.random.default_rng(case)
    xq, xs, wq, ws, x, w = exact_case(rng, fmt, counts, N, K)
    pw = pack(ops, wq, ws, fmt, dev)
    off = offsets_of(counts)
    out = ops.grouped_linear(to_dev(xq, dev), pw, to_dev(off, dev), to_dev(xs, dev))
    bias = bf16_round(rng.integers(-8, 9, (len(counts), N)).astype(np.float64))
    out_b = ops.grouped_linear(to_dev(xq, dev), pw, to_dev(off, dev), to_dev(xs, dev), bias=to_bf16(bias, dev))
    ops.check()
    assert np.array_equal(f64(out), bf16_round(oracle.grouped(x, w, off)))
    assert np.array_equal(f64(out_b), bf16_round(oracle.grouped(x, w, off, bias)))


# K split over clusters of 2 to 8 CTAs, tiles of 16, 32 and 64 rows
SPLITS = [((1, 0, 3, 1, 0, 2, 1, 0), 512, 1152), ((1, 1, 1), 128, 1152), ((0, 3, 0), 128, 2048), ((1, 1, 1), 128, 4096),
          ((37, 63), 128, 4096), ((3, 40, 0, 20, 7), 128, 4096), ((99, 1), 512, 1152), ((50, 50), 256, 1152), ((100, 0), 256, 2048),
          ((14,) * 5, 384, 4096), ((0, 0, 70, 0, 0), 256, 4096), ((64, 1, 0, 0, 5), 1408, 2048), ((65, 35), 640, 1152),
          ((1, 99), 512, 2048), ((50, 50), 384, 4096), ((20, 20, 20), 512, 2048), ((1,) * 8, 256, 2048)]


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("counts,N,K", SPLITS)
def test_exact_sums_of_split_k(fmt, counts, N, K):
    dev = device()
    rng = np.random.default_rng(len(counts) * N + K)
    xq, xs, wq, ws, x, w = exact_case(rng, fmt, counts, N, K)
    off = offsets_of(counts)
    out = ops.grouped_linear(to_dev(xq, dev), pack(ops, wq, ws, fmt, dev), to_dev(off, dev), to_dev(xs, dev))
    ops.check()
    assert np.array_equal(f64(out), bf16_round(oracle.grouped(x, w, off)))


def test_exact_sums_of_a_ragged_k():
    """fp8_128 with a last block of 16 along K and of 8 along N."""
    dev = device()
    rng = np.random.default_rng(50)
    for counts in ([3, 0, 20], [70, 140, 0], [300, 1, 600]):
        off = offsets_of(counts)
        N, K, R = 264, 400, sum(counts)
        xv, wv = rng.integers(-2, 3, (R, K)).astype(np.float64), rng.integers(-2, 3, (3, N, K)).astype(np.float64)
        xs, ws = np.full((R, 4), 0.5, np.float32), np.full((3, 3, 4), 2.0, np.float32)
        pw = pack(ops, oracle.e4m3_encode(wv), ws, "fp8_128", dev)
        out = ops.grouped_linear(to_dev(oracle.e4m3_encode(xv), dev), pw, to_dev(off, dev), to_dev(xs, dev))
        assert np.array_equal(f64(out), bf16_round(oracle.grouped(xv, wv, off)))


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("counts,N,K", [([3, 0, 9, 1], 264, 512), ([40, 30, 0, 64], 520, 384), ([200, 0, 333, 7], 392, 512)])
def test_bf16_x_in_order_and_picked(fmt, counts, N, K):
    dev = device()
    rng = np.random.default_rng(sum(counts))
    R, E, T = sum(counts), len(counts), 37
    q, s, w = weights(rng, fmt, E, N, K)
    pw = pack(ops, q, s, fmt, dev)
    off = offsets_of(counts)
    x = bf16_round(rng.standard_normal((R, K)) * np.where(rng.random((R, K)) < 1e-3, 100.0, 1.0))
    out = ops.grouped_linear(to_bf16(x, dev), pw, to_dev(off, dev))
    ops.check()
    of_row = np.repeat(np.arange(E), counts)
    xf = fake(x, fmt)
    ref = oracle.grouped(xf, w, off)
    bound = np.concatenate([product_bound(xf[off[e]:off[e + 1]], w[e], ref[off[e]:off[e + 1]]) for e in range(E)])
    assert_product(out, ref, bound)
    xq, xs = codes(x, fmt)
    assert torch.equal(out, ops.grouped_linear(to_dev(xq, dev), pw, to_dev(off, dev), to_dev(xs, dev)))
    # rows picked by an index: the same token more than once, and tokens that are none
    tokens = bf16_round(rng.standard_normal((T, K)))
    rows = rng.integers(0, T, R).astype(np.int32)
    rows[::7] = -1
    rows[3] = T
    got = ops.grouped_linear(to_bf16(tokens, dev), pw, to_dev(off, dev), rows=to_dev(rows, dev))
    valid = (rows >= 0) & (rows < T)
    picked = np.where(valid[:, None], tokens[np.where(valid, rows, 0)], 0.0)
    assert torch.equal(got, ops.grouped_linear(to_bf16(picked, dev), pw, to_dev(off, dev)))
    assert (f64(got)[~valid] == 0).all() and of_row.size == R


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("T,R", [(1, 4099), (300, 4100), (1025, 4100), (1026, 4100)])
def test_many_rows_picked_from_few_tokens(fmt, T, R):
    """Both sides of the rule that quantises the tokens and picks their codes: the bytes are those of x[rows]."""
    dev = device()
    rng = np.random.default_rng(T)
    N, K = 136, 4096 if fmt == "mxfp8" else 4112
    q, s, _ = weights(rng, fmt, 3, N, K)
    pw = pack(ops, q, s, fmt, dev)
    x = to_bf16(bf16_round(rng.standard_normal((T, K))), dev)
    rows = torch.from_numpy(rng.integers(-2, T + 2, R).astype(np.int32)).to(dev)
    off = torch.tensor([0, 1500, 1500, R - 3], dtype=torch.int32, device=dev)
    out = ops.grouped_linear(x, pw, off, rows=rows)
    inside = (rows >= 0) & (rows < T)
    picked = torch.where(inside[:, None], x[rows.clamp(0, T - 1).long()], torch.zeros((), dtype=x.dtype, device=dev))
    want = ops.grouped_linear(picked, pw, off)
    band, need = 4096, ops.grouped_workspace_size(pw.fmt, 3, R, N, K, False)
    ws = torch.full((2 * band + need,), 0xA5, dtype=torch.uint8, device=dev)
    again = ops.grouped_linear(x, pw, off, rows=rows, workspace=ws[band:band + need])
    ops.check()
    assert torch.equal(out[:R - 3], want[:R - 3]) and torch.equal(again[:R - 3], want[:R - 3])
    assert (ws[:band] == 0xA5).all() and (ws[band + need:] == 0xA5).all()


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("R,first,last", [(40, 5, 33), (400, 1, 399), (100, 0, 0)])
def test_rows_of_no_expert_are_left(fmt, R, first, last):
    dev = device()
    rng = np.random.default_rng(R)
    E, N, K = 3, 136, 256
    off = np.array([first, (first + last) // 2, (first + last) // 2, last], dtype=np.int32)
    q, s, w = weights(rng, fmt, E, N, K)
    out = torch.full((R, N), 7.0, dtype=torch.bfloat16, device=dev)
    x = to_bf16(bf16_round(rng.standard_normal((R, K))), dev)
    x[last:] = float("nan")  # whatever stands behind the last row
    pw = pack(ops, q, s, fmt, dev)
    got = ops.grouped_linear(x, pw, to_dev(off, dev), out=out)
    assert got is out
    o = f64(out)
    assert (o[:first] == 7).all() and (o[last:] == 7).all() and np.isfinite(o[first:last]).all()
    alone = ops.grouped_linear(x[first:last].contiguous(), pw, to_dev(off - first, dev))
    assert torch.equal(out[first:last], alone)


@pytest.mark.parametrize("fmt", FMTS)
def test_offsets_that_are_none(fmt):
    """Each is taken as at least 0 and the one before it, and at most the rows there are."""
    dev = device()
    rng = np.random.default_rng(9)
    E, N, K, R = 4, 136, 256, 50
    q, s, w = weights(rng, fmt, E, N, K)
    x = bf16_round(rng.standard_normal((R, K)))
    pw = pack(ops, q, s, fmt, dev)
    off = np.array([-5, 10, 4, 30, 1 << 30], dtype=np.int32)
    band = 4096
    buf = torch.full((2 * band + 2 * R * N,), 0xA5, dtype=torch.uint8, device=dev)
    out = buf[band:band + 2 * R * N].view(torch.bfloat16).view(R, N)
    ops.grouped_linear(to_bf16(x, dev), pw, to_dev(off, dev), out=out)
    ops.check()
    assert (buf[:band] == 0xA5).all() and (buf[-band:] == 0xA5).all()
    xf = fake(x, fmt)
    o = f64(out)
    for lo, hi, e in [(0, 10, 0), (10, 30, 2), (30, 50, 3)]:
        ref = xf[lo:hi] @ w[e].T
        assert (np.abs(o[lo:hi] - ref) <= product_bound(xf[lo:hi], w[e], ref)).all()
    # offsets that go up and down: no more work than the rows there are, for every kernel
    for rows in (8, 30, 200, 700):
        up_down = np.array([0, rows, 0, rows, 0], dtype=np.int32)
        x2 = to_bf16(bf16_round(rng.standard_normal((rows, K))), dev)
        got = ops.grouped_linear(x2, pw, to_dev(up_down, dev))
        ops.check()
        assert torch.equal(got, ops.grouped_linear(x2, pw, to_dev(np.array([0] + [rows] * 4, dtype=np.int32), dev)))


@pytest.mark.parametrize("fmt", FMTS)
def test_canary_bands(fmt):
    dev = device()
    rng = np.random.default_rng(6)
    band = 4096
    for counts, N, K in [([1, 0, 3], 136, 256), ([20, 40, 3], 264, 384), ([90, 110], 392, 256), ([300, 0, 500], 264, 384)]:
        R, E = sum(counts), len(counts)
        q, s, _ = weights(rng, fmt, E, N, K)
        pw = pack(ops, q, s, fmt, dev)
        x = to_bf16(bf16_round(rng.standard_normal((R, K))), dev)
        off = to_dev(offsets_of(counts), dev)
        need = ops.grouped_workspace_size(pw.fmt, E, R, N, K, False)
        outs = torch.full((2 * band + 2 * R * N,), 0xA5, dtype=torch.uint8, device=dev)
        wsb = torch.full((2 * band + need,), 0xA5, dtype=torch.uint8, device=dev)
        out = outs[band:band + 2 * R * N].view(torch.bfloat16).view(R, N)
        ops.grouped_linear(x, pw, off, out=out, workspace=wsb[band:band + need])
        ops.check()
        for t, n in ((outs, 2 * R * N), (wsb, need)):
            assert (t[:band] == 0xA5).all() and (t[band + n:] == 0xA5).all()
        assert torch.equal(out, ops.grouped_linear(x, pw, off))


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("R", [12, 90, 700])
def test_captured_graph_follows_the_offsets(fmt, R):
    dev = device()
    rng = np.random.default_rng(R)
    E, N, K = 6, 264, 512
    q, s, _ = weights(rng, fmt, E, N, K)
    pw = pack(ops, q, s, fmt, dev)
    splits = [rng.multinomial(R, rng.dirichlet(np.ones(E))) for _ in range(4)]
    offs = [to_dev(offsets_of(c), dev) for c in splits]
    xs = [to_bf16(bf16_round(rng.standard_normal((R, K))), dev) for _ in range(4)]
    want = [ops.grouped_linear(x, pw, o) for x, o in zip(xs, offs)]
    x, o = xs[0].clone(), offs[0].clone()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = ops.grouped_linear(x, pw, o)
    for i in (2, 0, 3, 1):
        x.copy_(xs[i])
        o.copy_(offs[i])
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want[i])
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [[], []]
    for _ in range(6):
        for i, st in enumerate(streams):
            with torch.cuda.stream(st):
                got[i].append(ops.grouped_linear(xs[i], pw, offs[i]))
    torch.cuda.synchronize()
    ops.check()
    for i in range(2):
        assert all(torch.equal(y, want[i]) for y in got[i])


def test_rows_past_31_bits_of_elements():
    """Output and input offsets past 2^31 elements: the last rows of a long batch are those of a short one."""
    dev = device()
    rng = np.random.default_rng(11)
    E, N, K = 3, 4096, 128
    R = (1 << 31) // N + 1000
    q, s, _ = weights(rng, "fp8_128", E, N, K)
    pw = pack(ops, q, s, "fp8_128", dev)
    x = torch.randn(R, K, device=dev).to(torch.bfloat16)
    off = to_dev(np.array([0, R // 2, R - 300, R], dtype=np.int32), dev)
    out = ops.grouped_linear(x, pw, off)
    ops.check()
    tail = ops.grouped_linear(x[R - 700:].contiguous(), pw, to_dev(np.array([0, 0, 400, 700], dtype=np.int32), dev))
    assert torch.equal(out[R - 700:], tail)


@pytest.mark.parametrize("fmt", FMTS)
def test_many_small_last_tiles_back_to_back(fmt):
    """Groups whose last tile holds a few rows, so that one CTA of a pair has none of them, next to full
    ones, many calls in a row: the pipelines of the two CTAs stay together."""
    dev = device()
    rng = np.random.default_rng(12)
    counts = [242, 266, 258, 235, 251, 261, 246, 258, 278, 263, 1, 513] * 3
    E, N, K, R = len(counts), 1024, 1024, sum(counts)
    wq = torch.randint(0, 100, (E, N, K), dtype=torch.uint8, device=dev)
    ws = (torch.rand(E, N // 128, K // 128, device=dev) + 0.5 if fmt == "fp8_128" else
          torch.randint(120, 130, (E, N, K // 32), dtype=torch.uint8, device=dev))
    pw = ops.process_weights_fp8_128(wq, ws) if fmt == "fp8_128" else ops.process_weights(wq, ws)
    x = to_bf16(bf16_round(rng.standard_normal((R, K))), dev)
    off = to_dev(offsets_of(counts), dev)
    want = ops.grouped_linear(x, pw, off)
    ops.check()
    for _ in range(5):
        outs = [ops.grouped_linear(x, pw, off) for _ in range(20)]
        ops.check()
        assert all(torch.equal(o, want) for o in outs)
    lo, hi = 242 + 266, 242 + 266 + 258
    alone = ops.grouped_linear(x[lo:hi].contiguous(), pw, to_dev(np.array([0, 0, 0] + [258] * (E - 2), dtype=np.int32), dev))
    assert torch.equal(want[lo:hi], alone)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("counts,N,K", [((1, 0, 3, 1, 2), 512, 1152), ((9, 40, 0, 20), 392, 1024), ((300, 0, 129, 700), 520, 640),
                                        ((1100, 64, 0, 900), 392, 1152)])
def test_beside_kernels_that_hold_the_sms(fmt, counts, N, K):
    """Warps that come late (the SMs are shared with another stream's kernels) meet every wait in time."""
    dev = device()
    rng = np.random.default_rng(N)
    q, s, _ = weights(rng, fmt, len(counts), N, K)
    pw, off = pack(ops, q, s, fmt, dev), to_dev(offsets_of(counts), dev)
    x = to_bf16(bf16_round(rng.standard_normal((sum(counts), K))), dev)
    xq, xs = ops.quantize_fp8_128(x) if fmt == "fp8_128" else ops.quantize(x)
    want = ops.grouped_linear(x, pw, off)
    other, st = torch.rand(1 << 24, device=dev), torch.cuda.Stream()
    torch.cuda.synchronize()
    outs = []
    for _ in range(20):
        for _ in range(4):
            other = torch.sin(other)
        with torch.cuda.stream(st):
            outs += [ops.grouped_linear(x, pw, off) for _ in range(5)] + [ops.grouped_linear(xq, pw, off, xs) for _ in range(5)]
    torch.cuda.synchronize()
    ops.check()
    assert all(torch.equal(o, want) for o in outs)
