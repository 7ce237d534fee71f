"""The block-128 FP8 quantiser and linear layer against the fp64 oracle."""

import numpy as np
import pytest
import torch

import oracle
from _grouped import assert_product, bf16_round, codes, f64, fake, product_bound, to_bf16, to_dev, weights
from _helpers import device
from mxfp8_block_scaled_02_gb300 import ops

pytestmark = pytest.mark.gpu


def all_patterns() -> np.ndarray:
    """Every finite bf16 value twice over, in blocks of like magnitude and in blocks of any."""
    bits = np.arange(65536, dtype=np.uint32)
    v = (bits << 16).view(np.float32).astype(np.float64)
    v = v[np.isfinite(v)]
    v = np.concatenate([v[np.argsort(np.abs(v), kind="stable")], np.random.default_rng(0).permutation(v)])
    return v[:v.size // 128 * 128].reshape(-1, 128)


def assert_codes(q: torch.Tensor, s: torch.Tensor, x: np.ndarray) -> None:
    want_q, want_s = oracle.quantize_b128(x)
    assert np.array_equal(s.cpu().numpy(), want_s, equal_nan=True)
    # below 2^-110 / 448 the scale keeps fewer bits, the codes do not depend on it
    assert np.array_equal(q.cpu().numpy(), want_q)


@pytest.mark.parametrize("rows,K", [(1, 16), (1, 128), (3, 144), (130, 496), (5, 4112), (257, 512), (2, 14336)])
def test_quantize_matches_the_oracle_bit_for_bit(rows, K):
    dev = device()
    rng = np.random.default_rng(rows * 1000 + K)
    x = bf16_round(rng.standard_normal((rows, K)) * np.exp2(rng.integers(-60, 60, (rows, 1))))
    x[rng.random(x.shape) < 0.01] *= 64
    x = bf16_round(x)
    assert_codes(*ops.quantize_fp8_128(to_bf16(x, dev)), x)


def test_quantize_every_bf16_value():
    dev = device()
    x = all_patterns()
    assert_codes(*ops.quantize_fp8_128(to_bf16(x, dev)), x)


def test_quantize_ties():
    """Quotients that are ties of two codes: amax and x with 448 x / amax = odd / 2^n, exactly."""
    dev = device()
    rng = np.random.default_rng(1)
    rows = []
    for odd in range(1, 16, 2):
        amax = 7.0 * odd  # s = odd / 64
        ties = np.array([c * odd for c in range(17, 32, 2) if c * odd < 256], dtype=np.float64)
        if ties.size:
            row = rng.choice(ties, 128) * np.exp2(-rng.integers(2, 9, 128)) * rng.choice([-1.0, 1.0], 128)
            row = np.where(np.abs(row) > amax, row / 64, row)
            row[0] = amax
            rows.append(row)
    x = np.array(rows)
    assert np.array_equal(x, bf16_round(x))
    assert_codes(*ops.quantize_fp8_128(to_bf16(x, dev)), x)


def test_quantize_special_blocks():
    dev = device()
    x = np.zeros((6, 256))
    x[1, 3] = -0.0
    x[2, 7] = np.inf
    x[3, 200] = np.nan
    x[4, :] = 2.0 ** -133
    x[5, 128:] = 3.0e38
    x = bf16_round(x)
    q, s = ops.quantize_fp8_128(to_bf16(x, dev))
    assert_codes(q, s, x)
    assert q[1, 3] == 0x80


@pytest.mark.parametrize("B,N,K", [(1, 128, 128), (1, 8, 16), (2, 136, 272), (3, 520, 1040)])
def test_quantize_weights(B, N, K):
    dev = device()
    w = bf16_round(np.random.default_rng(N).standard_normal((B, N, K)))
    q, s = ops.quantize_weights_fp8_128(to_bf16(w, dev))
    want_q, want_s = oracle.quantize_weights_b128(w)
    assert np.array_equal(s.cpu().numpy(), want_s) and np.array_equal(q.cpu().numpy(), want_q)
    q2, s2 = ops.quantize_weights_fp8_128(to_bf16(w[0], dev))
    assert torch.equal(q2, q[0]) and torch.equal(s2, s[0])


@pytest.mark.parametrize("merged", [True, False])
@pytest.mark.parametrize("rows,K", [(1, 16), (7, 144), (130, 1024)])
def test_silu_mul(rows, K, merged):
    """Within (6 + 1.2 |gate|) 2^-23 of y, then one E4M3 rounding: half a step is 2^-4 of a
    normal code and 2^-10 of the scale below; a scale's own error is that of its y, and 2^-23."""
    dev = device()
    rng = np.random.default_rng(rows + K)
    gate, up = bf16_round(3 * rng.standard_normal((rows, K))), bf16_round(3 * rng.standard_normal((rows, K)))
    if merged:
        q, s = ops.silu_mul_quantize(to_bf16(np.concatenate([gate, up], -1), dev), fmt="fp8_128")
    else:
        wide = to_bf16(np.concatenate([gate, np.zeros((rows, 16))], -1), dev)[:, :K]  # strided rows
        q, s = ops.silu_mul_quantize(wide, to_bf16(up, dev), fmt="fp8_128")
    y = gate / (1 + np.exp(-gate)) * up
    rel = (8 + 1.2 * np.abs(gate)) * 2.0 ** -23
    _, want_s = oracle.quantize_b128(y)
    top = np.repeat(want_s.astype(np.float64), 128, -1)[:, :K]
    worst = rel.max()
    assert (np.abs(f64(s) - want_s) <= want_s * worst).all()
    got = oracle.dequantize_b128(q.cpu().numpy(), s.cpu().numpy())
    half = np.maximum(np.abs(y) * 2.0 ** -4, top * 2.0 ** -10)
    assert (np.abs(got - y) <= half * (1 + 4 * worst) + np.abs(y) * worst).all()


def exact_case(rng, rows, N, K, B=None):
    """Codes and power-of-two scales whose products add up exactly in fp32, and to a bf16 value's
    rounding that is unique: small whole numbers, few of them not 0."""
    lead = () if B is None else (B,)
    xv = rng.integers(-2, 3, (*lead, rows, K)) * (rng.random((*lead, rows, K)) < 0.5)
    wv = rng.integers(-2, 3, (*lead, N, K)) * (rng.random((*lead, N, K)) < 0.5)
    xs = np.exp2(rng.integers(-2, 3, (*lead, rows, -(-K // 128)))).astype(np.float32)
    ws = np.exp2(rng.integers(-2, 3, (*lead, -(-N // 128), -(-K // 128)))).astype(np.float32)
    xq, wq = oracle.e4m3_encode(xv.astype(np.float64)), oracle.e4m3_encode(wv.astype(np.float64))
    ref = oracle.dequantize_b128(xq, xs) @ oracle.dequantize_weights_b128(wq, ws).swapaxes(-1, -2)
    return xq, xs, wq, ws, ref


# one row to several tiles; N and K that end inside a tile; both sides of the rules that pick a kernel
SHAPES = [(1, 8, 16), (1, 128, 128), (1, 4096, 512), (2, 264, 400), (16, 1000, 4112), (17, 256, 256), (31, 136, 1152),
          (33, 520, 784), (64, 384, 2048), (65, 128, 640), (100, 1000, 272), (128, 2056, 384), (129, 128, 128),
          (257, 392, 400), (300, 1032, 1040), (515, 776, 4112), (1030, 264, 528)]


@pytest.mark.parametrize("M,N,K", SHAPES)
def test_exact_sums(M, N, K):
    dev = device()
    rng = np.random.default_rng(M * 7 + N * 3 + K)
    xq, xs, wq, ws, ref = exact_case(rng, M, N, K)
    pw = ops.process_weights_fp8_128(to_dev(wq, dev), to_dev(ws, dev))
    out = ops.linear_fp8_128(to_dev(xq, dev), pw, x_scale=to_dev(xs, dev))
    ops.check()
    assert np.array_equal(f64(out), bf16_round(ref))
    bias = bf16_round(rng.integers(-8, 9, N).astype(np.float64))
    out = ops.linear_fp8_128(to_dev(xq, dev), pw, to_bf16(bias, dev), to_dev(xs, dev))
    assert np.array_equal(f64(out), bf16_round(ref + bias))


# K split over clusters of 2 to 8 CTAs, tiles of 16, 32 and 64 rows
SPLITS = [(1, 3240, 1152), (1, 120, 1152), (1, 120, 2048), (1, 1560, 4096), (1, 1160, 4096), (1, 120, 4096), (9, 3240, 1152),
          (9, 120, 1152), (9, 120, 2048), (9, 120, 4096), (24, 3000, 2048), (24, 2040, 2048), (100, 504, 2048), (150, 120, 4096),
          (150, 120, 8192), (150, 200, 2048), (150, 200, 4096), (150, 1000, 1152), (200, 120, 4096), (200, 200, 1152),
          (200, 200, 4096), (200, 200, 8192), (200, 280, 4096), (200, 440, 1152), (200, 440, 2048), (200, 1080, 2048)]


@pytest.mark.parametrize("M,N,K", SPLITS)
def test_exact_sums_of_split_k(M, N, K):
    test_exact_sums(M, N, K)
    test_bf16_x(M, N, K, True)


@pytest.mark.parametrize("B,M,N,K", [(2, 1, 128, 256), (3, 40, 136, 400), (4, 130, 264, 384), (16, 9, 1000, 512), (2, 300, 520, 272)])
def test_batches(B, M, N, K):
    dev = device()
    rng = np.random.default_rng(B + M)
    xq, xs, wq, ws, ref = exact_case(rng, M, N, K, B)
    pw = ops.process_weights_fp8_128(to_dev(wq, dev), to_dev(ws, dev))
    out = ops.linear_fp8_128(to_dev(xq, dev), pw, x_scale=to_dev(xs, dev))
    ops.check()
    assert np.array_equal(f64(out), bf16_round(ref))


@pytest.mark.parametrize("M,N,K", [(1, 1000, 4112), (2, 8, 16), (3, 520, 2064), (4, 264, 8192), (5, 4096, 384), (7, 256, 512),
                                   (8, 1032, 1040), (9, 1032, 1040), (8, 20000, 256),
                                   (1, 20000, 1152), (3, 20000, 1152), (5, 40000, 528), (8, 20000, 1152), (48, 520, 1040), (120, 264, 784), (333, 1000, 4112)])
@pytest.mark.parametrize("with_bias", [False, True])
def test_bf16_x(M, N, K, with_bias):
    dev = device()
    rng = np.random.default_rng(M + N + K)
    q, s, w = weights(rng, "fp8_128", N, K)
    x = bf16_round(rng.standard_normal((M, K)) * np.where(rng.random((M, K)) < 1e-3, 100.0, 1.0))
    bias = bf16_round(rng.standard_normal(N)) if with_bias else None
    pw = ops.process_weights_fp8_128(to_dev(q, dev), to_dev(s, dev))
    xd = to_bf16(x, dev)
    out = ops.linear_fp8_128(xd, pw, None if bias is None else to_bf16(bias, dev))
    ops.check()
    xf = fake(x, "fp8_128")
    ref = xf @ w.T + (0 if bias is None else bias)
    assert_product(out, ref, product_bound(xf, w, ref))
    # the same bytes from a quantised x, and again
    xq, xs = codes(x, "fp8_128")
    assert torch.equal(out, ops.linear_fp8_128(to_dev(xq, dev), pw, None if bias is None else to_bf16(bias, dev), to_dev(xs, dev)))
    assert torch.equal(out, ops.linear_fp8_128(xd, pw, None if bias is None else to_bf16(bias, dev)))


def test_nan_scale_stays_in_its_row():
    dev = device()
    rng = np.random.default_rng(3)
    x = bf16_round(rng.standard_normal((40, 256)))
    x[11, 200] = np.inf
    q, s, w = weights(rng, "fp8_128", 136, 256)
    out = f64(ops.linear_fp8_128(to_bf16(x, dev), ops.process_weights_fp8_128(to_dev(q, dev), to_dev(s, dev))))
    bad = np.isnan(out)
    assert bad[11].all() and not np.delete(bad, 11, 0).any()


def test_leading_axes_views_and_outputs():
    dev = device()
    rng = np.random.default_rng(4)
    xq, xs, wq, ws, ref = exact_case(rng, 6, 136, 272)
    pw = ops.process_weights_fp8_128(to_dev(wq, dev).view(torch.float8_e4m3fn), to_dev(ws, dev))
    x3 = to_dev(xq, dev).view(2, 3, 272)
    out = torch.empty(2, 3, 136, dtype=torch.bfloat16, device=dev)
    got = ops.linear_fp8_128(x3, pw, x_scale=to_dev(xs, dev).view(2, 3, -1), out=out)
    assert got is out and np.array_equal(f64(out).reshape(6, 136), bf16_round(ref))
    # a view that does not start on 16 bytes is copied
    buf = torch.empty(xq.size + 3, dtype=torch.uint8, device=dev)
    odd = buf[3:].view(6, 272).copy_(to_dev(xq, dev))
    assert torch.equal(ops.linear_fp8_128(odd, pw, x_scale=to_dev(xs, dev)), out.view(6, 136))
    empty = ops.linear_fp8_128(torch.empty(0, 272, dtype=torch.bfloat16, device=dev), pw)
    assert tuple(empty.shape) == (0, 136)


def test_canary_bands():
    """Exactly the documented bytes of output, workspace and codes are written."""
    dev = device()
    rng = np.random.default_rng(6)
    band = 4096
    for M, N, K in [(1, 136, 400), (20, 264, 528), (100, 1000, 272), (300, 392, 400)]:
        q, s, _ = weights(rng, "fp8_128", N, K)
        pw = ops.process_weights_fp8_128(to_dev(q, dev), to_dev(s, dev))
        x = to_bf16(bf16_round(rng.standard_normal((M, K))), dev)
        need = ops.workspace_size_fp8_128(1, M, N, K, False)
        outs = torch.full((2 * band + 2 * M * N,), 0xA5, dtype=torch.uint8, device=dev)
        wsb = torch.full((2 * band + need,), 0xA5, dtype=torch.uint8, device=dev)
        out = outs[band:band + 2 * M * N].view(torch.bfloat16).view(M, N)
        ops.linear_fp8_128(x, pw, out=out, workspace=wsb[band:band + need])
        ops.check()
        for t, n in ((outs, 2 * M * N), (wsb, need)):
            assert (t[:band] == 0xA5).all() and (t[band + n:] == 0xA5).all()
        assert torch.equal(out, ops.linear_fp8_128(x, pw))


@pytest.mark.parametrize("M", [1, 40, 200])
def test_graph_and_streams(M):
    """A captured call follows its input's contents; calls on two streams with their own workspaces
    give the same as one after the other."""
    dev = device()
    rng = np.random.default_rng(7)
    q, s, _ = weights(rng, "fp8_128", 520, 784)
    pw = ops.process_weights_fp8_128(to_dev(q, dev), to_dev(s, dev))
    xs = [to_bf16(bf16_round(rng.standard_normal((M, 784))), dev) for _ in range(4)]
    want = [ops.linear_fp8_128(x, pw) for x in xs]
    x = xs[0].clone()
    ops.linear_fp8_128(x, pw)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = ops.linear_fp8_128(x, pw)
    for i in (2, 1, 3):
        x.copy_(xs[i])
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want[i])
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = [[], []]
    for _ in range(8):
        for i, st in enumerate(streams):
            with torch.cuda.stream(st):
                outs[i].append(ops.linear_fp8_128(xs[i], pw))
    torch.cuda.synchronize()
    ops.check()
    for i in range(2):
        assert all(torch.equal(o, want[i]) for o in outs[i])


@pytest.mark.parametrize("M", [1, 20, 40, 100])
def test_beside_kernels_that_hold_the_sms(M):
    """Warps that come late (the SMs are shared with another stream's kernels) meet every wait in time."""
    dev = device()
    rng = np.random.default_rng(M)
    q, s, _ = weights(rng, "fp8_128", 1000, 1040)
    pw = ops.process_weights_fp8_128(to_dev(q, dev), to_dev(s, dev))
    x = to_bf16(bf16_round(rng.standard_normal((M, 1040))), dev)
    xq, xs = ops.quantize_fp8_128(x)
    want = ops.linear_fp8_128(x, pw)
    other, st = torch.rand(1 << 24, device=dev), torch.cuda.Stream()
    torch.cuda.synchronize()
    outs = []
    for _ in range(20):
        for _ in range(4):
            other = torch.sin(other)
        with torch.cuda.stream(st):
            outs += [ops.linear_fp8_128(x, pw) for _ in range(5)] + [ops.linear_fp8_128(xq, pw, x_scale=xs) for _ in range(5)]
    torch.cuda.synchronize()
    ops.check()
    assert all(torch.equal(o, want) for o in outs)


@pytest.mark.parametrize("what", ["quantised x", "bias"])
def test_inputs_the_kernel_ahead_has_just_written(what):
    """x from the quantise call and the bias from a few-token product, back to back, many times."""
    dev = device()
    rng = np.random.default_rng(8)
    q, s, _ = weights(rng, "fp8_128", 264, 512)
    pw = ops.process_weights_fp8_128(to_dev(q, dev), to_dev(s, dev))
    x = to_bf16(bf16_round(rng.standard_normal((24, 512))), dev)
    if what == "bias":
        first = ops.linear_fp8_128(x[:1], pw)
        want = ops.linear_fp8_128(x, pw, first.view(264).clone())
        torch.cuda.synchronize()
        for _ in range(50):
            got = ops.linear_fp8_128(x, pw, ops.linear_fp8_128(x[:1], pw).view(264))
            assert torch.equal(got, want)
    else:
        want = ops.linear_fp8_128(x, pw)
        for _ in range(50):
            xq, xs = ops.quantize_fp8_128(x)
            assert torch.equal(ops.linear_fp8_128(xq, pw, x_scale=xs), want)
