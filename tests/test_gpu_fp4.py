"""4-bit quantisation and product (MXFP4, NVFP4) against the fp64 oracle."""

import numpy as np
import pytest
import torch

import oracle
from _helpers import bf16_to_dev, device, u8_to_dev
from mxfp8_block_scaled_02_gb300 import ops, synth

pytestmark = pytest.mark.gpu
FMTS = ["mxfp4", "nvfp4"]


def bf16_bits_of(x):
    return (torch.from_numpy(np.ascontiguousarray(x)).float().to(torch.bfloat16).view(torch.int16).numpy().view(np.uint16))


def rand_bf16(rng, *shape, scale=1.0):
    bits = bf16_bits_of(rng.standard_normal(shape) * scale)
    return bits, synth.bf16_bits_to_f64(bits)


def scale_tensor(g, dev):
    return None if g is None else torch.tensor([g], dtype=torch.float32, device=dev)


def atoms_of(s, K, fmt):
    """Row-major scale bytes [R, KB] -> (atom bytes, mask of the bytes a row writes, its padding included)."""
    R, KB = s.shape
    KT, RT = -(-KB // 4), -(-R // 128)
    out = np.zeros(KT * RT * 512, dtype=np.uint8)
    mask = np.zeros_like(out, dtype=bool)
    r = np.arange(R)[:, None]
    kb = np.arange(KT * 4)[None, :]
    off = ((kb // 4) * RT + r // 128) * 512 + (r % 32) * 16 + ((r // 32) % 4) * 4 + kb % 4
    padded = np.zeros((R, KT * 4), dtype=np.uint8)
    padded[:, :KB] = s
    out[off] = padded
    mask[off] = True
    return out, mask


# ---------------------------------------------------------------- quantise
@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("rows,K", [(1, 32), (3, 64), (130, 96), (5, 4128), (257, 512)])
def test_quantize_matches_the_oracle_bit_for_bit(fmt, rows, K):
    dev = device()
    rng = np.random.default_rng(rows * 1000 + K)
    bits, x = rand_bf16(rng, rows, K)
    x = x * np.exp2(rng.integers(-60, 40, size=(rows, K // 32)).repeat(32, axis=1) if fmt == "mxfp4" else 0.0)
    bits = bf16_bits_of(x)
    x = synth.bf16_bits_to_f64(bits)
    g = None if fmt == "mxfp4" else float(np.float32(np.abs(x).max() / 2688))
    codes, s = oracle.quantize4(x, fmt, g or 1.0)
    q_d, s_d = ops.quantize_fp4(bf16_to_dev(bits, dev), fmt, tensor_scale=scale_tensor(g, dev))
    assert np.array_equal(s_d.cpu().numpy(), s)
    assert np.array_equal(q_d.cpu().numpy(), oracle.pack(codes))
    pa = ops.quantize_packed_fp4(bf16_to_dev(bits, dev), 1, fmt, tensor_scale=scale_tensor(g, dev))
    want, mask = atoms_of(s, K, fmt)
    assert np.array_equal(pa.x_q.cpu().numpy().reshape(rows, -1), oracle.pack(codes))
    assert np.array_equal(pa.sf_packed.cpu().numpy()[mask], want[mask])


@pytest.mark.parametrize("fmt", FMTS)
def test_quantize_ties_zeros_subnormals_and_nonfinite_blocks(fmt):
    dev = device()
    n = ops.QBLOCK[fmt]
    rows = [np.resize([0.25, -0.75, 1.25, 1.75, 2.5, -3.5, 5.0, 7.0], n),   # every tie, and saturation
            np.zeros(n), np.full(n, -0.0), np.resize([1e-39, -2e-40], n), np.resize([3e38, 1.0], n),
            np.resize([1.0, np.inf], n), np.resize([np.nan, 2.0], n), np.resize([-np.inf, 0.0], n)]
    x = np.concatenate(rows + rows)[None, :]
    x = np.resize(x, (1, -(-x.shape[1] // 32) * 32))
    with np.errstate(over="ignore"):
        bits = bf16_bits_of(x)
    x = synth.bf16_bits_to_f64(bits)
    codes, s = oracle.quantize4(x, fmt, 1.0)
    q_d, s_d = ops.quantize_fp4(bf16_to_dev(bits, dev), fmt)
    assert np.array_equal(s_d.cpu().numpy(), s)
    assert np.array_equal(q_d.cpu().numpy(), oracle.pack(codes))


def test_unpack_covers_every_byte():
    dev = device()
    q = np.arange(256, dtype=np.uint8).reshape(4, 64)
    got = ops.unpack_fp4(u8_to_dev(q, dev)).float().cpu().numpy()
    want = oracle.e2m1_value(oracle.unpack(q))
    assert np.array_equal(got, want) and np.array_equal(np.signbit(got), np.signbit(want))


def test_mxfp4_weights_serve_the_mxfp8_layer_after_unpacking():
    dev = device()
    rng = np.random.default_rng(3)
    wb, _ = rand_bf16(rng, 256, 512, scale=0.05)
    wq, ws = ops.quantize_fp4(bf16_to_dev(wb, dev), "mxfp4")
    pw8 = ops.process_weights(ops.unpack_fp4(wq), ws)
    xb, x = rand_bf16(rng, 20, 512)
    w = oracle.dequantize4(oracle.unpack(wq.cpu().numpy()), ws.cpu().numpy(), "mxfp4")
    xq, xs = oracle.quantize(x)
    ref = oracle.dequantize(xq, xs) @ w.T
    got = ops.linear(bf16_to_dev(xb, dev), pw8).double().cpu().numpy()
    bound = 2.0 ** -8 * np.abs(ref) + 1e-5 * (np.abs(oracle.dequantize(xq, xs)) @ np.abs(w).T)
    assert (np.abs(got - ref) <= bound).all()


# ---------------------------------------------------------------- product
def small_operand(rng, fmt, B, R, K):
    """Codes and power-of-two scales in {1/2, 1, 2}: every product is a multiple
    of 1/16 and the sums stay far below 2^24 / 16, so fp32 adds them exactly in any order."""
    codes = rng.integers(0, 16, size=(B, R, K), dtype=np.uint8)
    KB = K // ops.QBLOCK[fmt]
    pick = rng.integers(0, 3, size=(B, R, KB))
    s = (126 + pick if fmt == "mxfp4" else 0x30 + 8 * pick).astype(np.uint8)
    return codes, s


def to_bf16_f64(x):
    return torch.from_numpy(x).to(torch.float32).to(torch.bfloat16).double().numpy()


SHAPES = [(1, 1, 8, 32), (1, 5, 264, 64), (1, 129, 256, 96), (1, 16, 1000, 4128), (1, 128, 520, 1312),
          (1, 300, 72, 544), (1, 600, 1288, 288), (3, 70, 136, 160), (2, 257, 264, 1056), (1, 64, 4096, 1024),
          (1, 33, 2056, 2080), (1, 100, 4104, 512)]


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("B,M,N,K", SHAPES)
def test_product_is_exact_on_exact_sums(fmt, B, M, N, K):
    dev = device()
    rng = np.random.default_rng(B + 7 * M + 11 * N + K)
    xc, xs = small_operand(rng, fmt, B, M, K)
    wc, ws = small_operand(rng, fmt, B, N, K)
    x64 = oracle.dequantize4(xc, xs, fmt)
    w64 = oracle.dequantize4(wc, ws, fmt)
    ref = to_bf16_f64(np.einsum("bmk,bnk->bmn", x64, w64, optimize=True))
    sq = (lambda a: a) if B > 1 else (lambda a: a[0])
    pw = ops.process_weights_fp4(u8_to_dev(sq(oracle.pack(wc)), dev), u8_to_dev(sq(ws), dev), fmt)
    got = ops.linear_fp4(u8_to_dev(sq(oracle.pack(xc)), dev), pw, x_scale=u8_to_dev(sq(xs), dev))
    ops.check()
    assert np.array_equal(got.double().cpu().numpy(), sq(ref))


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("B,M,N,K", SHAPES)
def test_linear_on_bf16_against_the_oracle(fmt, B, M, N, K):
    """|out - ref| <= 2^-8 |ref| (one bf16 rounding, with room) + (K / 16 + 16) 2^-23 S, where S is the
    sum of the products' magnitudes: fp32 sums of K / 64 steps, each step's terms aligned to fp32."""
    dev = device()
    rng = np.random.default_rng(2 * B + 5 * M + 3 * N + K)
    xb, x = rand_bf16(rng, B, M, K)
    wb, w = rand_bf16(rng, B, N, K, scale=0.02)
    bb, bias = rand_bf16(rng, N, scale=0.1)
    gx, gw = (None, None) if fmt == "mxfp4" else [float(np.float32(np.abs(a).max() / 2688)) for a in (x, w)]
    xd = oracle.dequantize4(*oracle.quantize4(x, fmt, gx or 1.0), fmt, gx or 1.0)
    wd = oracle.dequantize4(*oracle.quantize4(w, fmt, gw or 1.0), fmt, gw or 1.0)
    ref = np.einsum("bmk,bnk->bmn", xd, wd, optimize=True) + bias
    mag = np.einsum("bmk,bnk->bmn", np.abs(xd), np.abs(wd), optimize=True) + np.abs(bias)
    bound = 2.0 ** -8 * np.abs(ref) + (K / 16 + 16) * 2.0 ** -23 * mag
    sq = (lambda a: a) if B > 1 else (lambda a: a[0])
    xt, wt, bt = bf16_to_dev(sq(xb), dev), bf16_to_dev(sq(wb), dev), bf16_to_dev(bb, dev)
    tx, tw = scale_tensor(gx, dev), scale_tensor(gw, dev)
    wq, ws = ops.quantize_fp4(wt, fmt, tensor_scale=tw)
    pw = ops.process_weights_fp4(wq, ws, fmt, tensor_scale=tw)
    got = ops.linear_fp4(xt, pw, bt, tensor_scale=tx)
    ops.check()
    assert (np.abs(got.double().cpu().numpy() - sq(ref)) <= sq(bound)).all()
    # the other forms of the same call
    xq, xs = ops.quantize_fp4(xt, fmt, tensor_scale=tx)
    codes = ops.linear_fp4(xq, pw, bt, xs, tensor_scale=tx)
    packed = ops.gemm_packed_fp4(ops.quantize_packed_fp4(xt, B, fmt, tensor_scale=tx), pw, bt)
    ops.check()
    for other in (codes, packed.view(got.shape)):
        assert (np.abs(other.double().cpu().numpy() - sq(ref)) <= sq(bound)).all()
    assert torch.equal(got, ops.linear_fp4(xt, pw, bt, tensor_scale=tx))  # the same on every call


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("M,N,K", [(1, 4096, 4096), (3, 264, 96), (7, 1000, 4128), (12, 136, 8224), (13, 520, 2080),
                                   (16, 72, 14336), (16, 14336, 512)])
def test_few_tokens_are_quantised_inside_to_the_same_bytes(fmt, M, N, K):
    """Up to 16 bf16 rows are quantised in the product's own kernel: the output is bit for bit that of the codes
    the quantise call gives, whatever a block holds."""
    dev = device()
    rng = np.random.default_rng(M + N + K)
    x = rand_bf16(rng, M, K)[1] * np.exp2(rng.integers(-8, 9, size=(M, K // 32)).repeat(32, axis=1))
    x[M // 2, :32] = 0.0
    x[0, K - 1] = np.inf
    xt = bf16_to_dev(bf16_bits_of(x), dev)
    wt = bf16_to_dev(rand_bf16(rng, N, K)[0], dev)
    g = scale_tensor(None if fmt == "mxfp4" else 0.37, dev)
    pw = ops.process_weights_fp4(*ops.quantize_fp4(wt, fmt), fmt)
    inside = ops.linear_fp4(xt, pw, tensor_scale=g)
    q, s = ops.quantize_fp4(xt, fmt, tensor_scale=g)
    codes = ops.linear_fp4(q, pw, x_scale=s, tensor_scale=g)
    ops.check()
    assert torch.equal(inside.view(torch.int16), codes.view(torch.int16))
    assert torch.isnan(inside[0]).all() and torch.isfinite(inside[1:]).all()


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("M", [20, 200])
def test_nan_blocks_stay_in_their_row_and_column(fmt, M):
    dev = device()
    rng = np.random.default_rng(M)
    N, K = 264, 544
    xb, x = rand_bf16(rng, M, K)
    wb, w = rand_bf16(rng, N, K)
    x[7, 100], w[13, 543] = np.inf, np.nan
    xt, wt = bf16_to_dev(bf16_bits_of(x), dev), bf16_to_dev(bf16_bits_of(w), dev)
    pw = ops.process_weights_fp4(*ops.quantize_fp4(wt, fmt), fmt)
    out = ops.linear_fp4(xt, pw).float().cpu().numpy()
    bad = np.isnan(out)
    want = np.zeros_like(bad)
    want[7, :], want[:, 13] = True, True
    assert np.array_equal(bad, want)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("M", [9, 140])
def test_padding_rows_of_the_activation_scales_do_not_matter(fmt, M):
    """quantize_packed leaves the atoms' padding rows as they were; whatever they hold, the output is the same."""
    dev = device()
    rng = np.random.default_rng(5)
    N, K = 136, 352
    xt = bf16_to_dev(rand_bf16(rng, M, K)[0], dev)
    wt = bf16_to_dev(rand_bf16(rng, N, K)[0], dev)
    pw = ops.process_weights_fp4(*ops.quantize_fp4(wt, fmt), fmt)
    outs = []
    for fill in (0x00, 0xFF):
        pa = ops.quantize_packed_fp4(xt, 1, fmt)
        written = torch.zeros_like(pa.sf_packed)
        _, mask = atoms_of(np.zeros((M, K // ops.QBLOCK[fmt]), np.uint8), K, fmt)
        written = torch.from_numpy(mask).to(dev)
        pa.sf_packed[~written] = fill
        outs.append(ops.gemm_packed_fp4(pa, pw))
    assert torch.equal(outs[0], outs[1]) and torch.isfinite(outs[0]).all()


@pytest.mark.parametrize("M", [3, 90, 256])
def test_guard_bands_around_the_outputs_stay(M):
    dev = device()
    N, K = 1000, 416
    x = torch.randn(M, K, device=dev).to(torch.bfloat16)
    w = torch.randn(N, K, device=dev).to(torch.bfloat16)
    pw = ops.process_weights_fp4(*ops.quantize_fp4(w, "nvfp4"), "nvfp4")
    big = torch.full((M * N + 4096,), 7.0, dtype=torch.bfloat16, device=dev)
    ops.linear_fp4(x, pw, out=big[2048:2048 + M * N])
    ops.check()
    assert (big[:2048] == 7).all() and (big[2048 + M * N:] == 7).all()
    assert torch.equal(big[2048:2048 + M * N].view(M, N), ops.linear_fp4(x, pw))


def test_empty_calls():
    dev = device()
    w = torch.randn(64, 64, device=dev).to(torch.bfloat16)
    pw = ops.process_weights_fp4(*ops.quantize_fp4(w), "mxfp4")
    x = torch.empty(0, 64, dtype=torch.bfloat16, device=dev)
    assert ops.linear_fp4(x, pw).shape == (0, 64)
    q, s = ops.quantize_fp4(x)
    assert q.shape == (0, 32) and s.shape == (0, 2)
    assert ops.linear_fp4(q, pw, x_scale=s).shape == (0, 64)


def test_refusals():
    dev = device()
    x = torch.randn(4, 64, device=dev).to(torch.bfloat16)
    pw = ops.process_weights_fp4(*ops.quantize_fp4(x, "mxfp4"), "mxfp4")  # N = 4
    with pytest.raises(ops.MxStatusError, match="UNSUPPORTED"):
        ops.linear_fp4(x, pw)  # N % 8
    w = torch.randn(16, 64, device=dev).to(torch.bfloat16)
    pw = ops.process_weights_fp4(*ops.quantize_fp4(w, "mxfp4"), "mxfp4")
    g = torch.ones(1, device=dev)
    with pytest.raises(ValueError):
        ops.linear_fp4(x, pw, tensor_scale=g)  # mxfp4 has none
    with pytest.raises(ValueError):
        ops.quantize_fp4(x, "nvfp4", tensor_scale=g.half())
    with pytest.raises(ValueError):
        ops.quantize_fp4(x, "fp4")
    with pytest.raises(TypeError):
        ops.quantize_fp4(x.float())
    with pytest.raises(ops.MxStatusError, match="INVALID_ARG"):
        ops.quantize_fp4(x[:, :40].contiguous())  # K % 32
    with pytest.raises(ValueError):
        ops.linear_fp4(x[:, :32].contiguous(), pw)
    with pytest.raises(ValueError):
        ops.linear(x, pw)  # 8-bit entry points do not take 4-bit weights
    with pytest.raises(ValueError):
        ops.gemm_packed(ops.quantize_packed(x), pw)
    with pytest.raises(ValueError):
        ops.gemm_packed_fp4(ops.quantize_packed_fp4(x, 1, "nvfp4"), pw)
    with pytest.raises(ValueError):
        ops.save_packed(pw)
    with pytest.raises(ValueError):
        ops.linear_fp4(x, pw, torch.zeros(8, dtype=torch.bfloat16, device=dev))
    with pytest.raises(ValueError):
        ops.linear_fp4(x, pw, out=torch.empty(4, 8, dtype=torch.bfloat16, device=dev))
    with pytest.raises(ops.MxStatusError, match="workspace"):
        ops.linear_fp4(x.repeat(5, 1), pw, workspace=torch.empty(16, dtype=torch.uint8, device=dev))


def test_misaligned_views_are_taken():
    dev = device()
    buf = torch.randn(8 * 64 + 1, device=dev).to(torch.bfloat16)
    x = buf[1:].view(8, 64)
    q, s = ops.quantize_fp4(x, "nvfp4")
    q2, s2 = ops.quantize_fp4(x.clone(), "nvfp4")
    assert torch.equal(q, q2) and torch.equal(s, s2)


@pytest.mark.parametrize("fmt", FMTS)
def test_graph_capture_and_two_streams(fmt):
    dev = device()
    torch.manual_seed(1)
    pws = []
    for N, K in [(1024, 512), (264, 2048), (2048, 1024)]:
        w = torch.randn(N, K, device=dev).to(torch.bfloat16)
        pws.append(ops.process_weights_fp4(*ops.quantize_fp4(w, fmt), fmt))
    xs = [[torch.randn(m, p.K, device=dev).to(torch.bfloat16) for m in (1, 40, 100, 300)] for p in pws]

    def run():
        return [ops.linear_fp4(x, p) for p, row in zip(pws, xs) for x in row]

    ref = run()
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    got = []
    for s in (s1, s2, s1, s2):
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            got.append(run())
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = run()
    for x in [x for row in xs for x in row]:
        x.mul_(2.0)
    graph.replay()
    torch.cuda.synchronize()
    ops.check()
    for outs in got:
        assert all(torch.equal(a, b) for a, b in zip(ref, outs))
    # doubling x doubles an MXFP4 output exactly (scales are powers of two)
    if fmt == "mxfp4":
        assert all(torch.equal(2 * a, b) for a, b in zip(ref, captured))
    else:
        assert all(torch.equal(a, b) for a, b in zip(run(), captured))


@pytest.mark.parametrize("fmt", FMTS)
def test_outputs_past_two_billion_elements(fmt):
    """M N beyond 32 bits: the last rows equal the same rows multiplied alone (every tile sums K in the same order)."""
    dev = device()
    M, N, K = 140000, 16384, 128
    gen = torch.Generator(device=dev).manual_seed(2)
    x = torch.randn(M, K, device=dev, generator=gen).to(torch.bfloat16)
    w = torch.randn(N, K, device=dev, generator=gen).to(torch.bfloat16)
    pw = ops.process_weights_fp4(*ops.quantize_fp4(w, fmt), fmt)
    out = ops.linear_fp4(x, pw)
    tail = ops.linear_fp4(x[-300:].clone(), pw)
    ops.check()
    assert torch.equal(out[-300:], tail) and torch.equal(out[:300], ops.linear_fp4(x[:300].clone(), pw))
