"""RMS norm and gated activation with quantised outputs, and the gated MLP block, against fp64.

The kernels compute y in fp32 and round it once to its element.  A code or a
scale byte may then differ from the fp64 result's only where y lies within the
fp32 error of a rounding boundary: it must be the one that y (1 - d), y or
y (1 + d) rounds to.  d is the fp32 relative error of y: for the norm the sum
of K squares by threads of at most 64 terms, two trees of 5 steps and up to 32
partials ((64 + 10) 2^-24, halved by the root) plus four roundings and rsqrtf's
2 ulp; for the activation __expf (2 + |1.2 gate| ulp, |gate| <= 30 here), one
division (2 ulp) and three roundings.  Both stay below 1e-5.
"""

import numpy as np
import pytest
import torch

import oracle
from _helpers import bf16_to_dev, device
from mxfp8_block_scaled_02_gb300 import mlp, ops, synth
from test_gpu_fp4 import atoms_of, bf16_bits_of, rand_bf16, scale_tensor, to_bf16_f64

pytestmark = pytest.mark.gpu
D = 1e-5
FMTS = ["mxfp8", "mxfp4", "nvfp4"]
G = {"mxfp8": None, "mxfp4": None, "nvfp4": float(np.float32(0.0031))}


def unpacked(q, fmt):
    q = q.cpu().numpy()
    return q if fmt == "mxfp8" else oracle.unpack(q)


def check_quantised(codes, scales, y, fmt, what=""):
    """codes (one per byte) and row-major scale bytes of fp64 y."""
    g = G[fmt] or 1.0
    n = ops.QBLOCK[fmt]
    ok = np.zeros(codes.shape, dtype=bool)
    ok_s = np.zeros(scales.shape, dtype=bool)
    for f in (1 - D, 1.0, 1 + D):
        c, s = oracle.quantize_any(y * f, fmt, g)
        ok_s |= s == scales
        same_scale = np.repeat(s == scales, n, axis=-1)
        # the sign of a zero result does not matter
        zero = ((codes & 0x7F) == 0) & ((c & 0x7F) == 0) if fmt == "mxfp8" else ((codes & 7) == 0) & ((c & 7) == 0)
        ok |= same_scale & ((c == codes) | zero)
    assert ok_s.all(), f"{what}: {int((~ok_s).sum())} scale bytes"
    assert ok.all(), f"{what}: {int((~ok).sum())} codes of {codes.size}"


def packed_to_rows(pa, fmt):
    """Row-major scale bytes out of packed atoms, and the bytes that pad each row."""
    KB = pa.K // ops.QBLOCK[fmt]
    probe = np.arange(pa.M * KB).reshape(pa.M, KB)
    KT, RT = -(-KB // 4), -(-pa.M // 128)
    r, kb = np.arange(pa.M)[:, None], np.arange(KT * 4)[None, :]
    off = ((kb // 4) * RT + r // 128) * 512 + (r % 32) * 16 + ((r // 32) % 4) * 4 + kb % 4
    rows = pa.sf_packed.cpu().numpy()[off]
    del probe
    return rows[:, :KB], rows[:, KB:]


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("res", ["none", "bf16", "fp32"])
@pytest.mark.parametrize("M,K", [(1, 32), (3, 96), (130, 4128), (2, 8224), (1, 32768), (700, 512)])
def test_norm_against_fp64(fmt, res, M, K):
    dev = device()
    rng = np.random.default_rng(M + K + len(res))
    xb, x = rand_bf16(rng, M, K, scale=2.0)
    wb, w = rand_bf16(rng, K, scale=0.3)
    rt = r = None
    if res == "bf16":
        rb, r = rand_bf16(rng, M, K, scale=3.0)
        rt = bf16_to_dev(rb, dev)
    elif res == "fp32":
        rt = torch.from_numpy((rng.standard_normal((M, K)) * 3.0).astype(np.float32)).to(dev)
        r = rt.cpu().numpy().astype(np.float64)
    y_out = torch.empty(M, K, dtype=torch.bfloat16, device=dev)
    g = scale_tensor(G[fmt], dev)
    args = dict(eps=1e-5, fmt=fmt, tensor_scale=g)
    (q, s), t_out = ops.rmsnorm_quantize(bf16_to_dev(xb, dev), bf16_to_dev(wb, dev), rt, y=y_out, **args)
    t, y = oracle.rmsnorm(x, w, r, 1e-5)
    check_quantised(unpacked(q, fmt), s.cpu().numpy(), y, fmt)
    got_y = y_out.double().cpu().numpy()
    assert (np.abs(got_y - y) <= (2.0 ** -8 + D) * np.abs(y)).all()
    if res == "none":
        assert t_out is None
    else:
        t32 = x.astype(np.float32) + r.astype(np.float32)
        want = to_bf16_f64(t32.astype(np.float64)) if res == "bf16" else t32.astype(np.float64)
        assert t_out.dtype == rt.dtype and np.array_equal(t_out.double().cpu().numpy(), want)
    pa, _ = ops.rmsnorm_quantize(bf16_to_dev(xb, dev), bf16_to_dev(wb, dev), rt, packed=True, **args)
    rows, pad = packed_to_rows(pa, fmt)
    assert torch.equal(pa.x_q.view(M, -1), q) and np.array_equal(rows, s.cpu().numpy()) and not pad.any()


@pytest.mark.parametrize("fmt", FMTS)
def test_norm_in_place_strided_and_leading_axes(fmt):
    dev = device()
    torch.manual_seed(2)
    wide = torch.randn(6, 5, 640, device=dev).to(torch.bfloat16)
    w = torch.randn(256, device=dev).to(torch.bfloat16)
    res = torch.randn(6, 5, 256, device=dev)
    g = scale_tensor(G[fmt], dev)
    x = wide[..., 128:384]
    (q0, s0), t0 = ops.rmsnorm_quantize(x.contiguous(), w, res, fmt=fmt, tensor_scale=g)
    for view in (x, wide[..., 128:384].transpose(0, 1).contiguous().transpose(0, 1)):
        (q, s), t = ops.rmsnorm_quantize(view, w, res, fmt=fmt, tensor_scale=g)
        assert q.shape[:2] == (6, 5) and torch.equal(q, q0) and torch.equal(s, s0) and torch.equal(t, t0)
    odd = wide.view(-1)[3:3 + 30 * 256].view(6, 5, 256)  # rows not on 16-byte boundaries
    (q, s), _ = ops.rmsnorm_quantize(odd, w, fmt=fmt, tensor_scale=g)
    (q1, s1), _ = ops.rmsnorm_quantize(odd.clone(), w, fmt=fmt, tensor_scale=g)
    assert torch.equal(q, q1) and torch.equal(s, s1)
    inplace = res.clone()
    (q, s), t = ops.rmsnorm_quantize(x, w, inplace, fmt=fmt, tensor_scale=g, residual_out=inplace)
    assert t.data_ptr() == inplace.data_ptr() and torch.equal(inplace, t0) and torch.equal(q, q0)
    bigres = torch.randn(30, 512, device=dev).to(torch.bfloat16)  # a strided residual
    (qa, _), ta = ops.rmsnorm_quantize(x.reshape(30, 256), w, bigres[:, 256:], fmt=fmt, tensor_scale=g)
    (qb, _), tb = ops.rmsnorm_quantize(x.reshape(30, 256), w, bigres[:, 256:].contiguous(), fmt=fmt, tensor_scale=g)
    assert torch.equal(qa, qb) and torch.equal(ta, tb)


@pytest.mark.parametrize("fmt", FMTS)
def test_norm_zero_rows_and_nonfinite_rows(fmt):
    dev = device()
    x = torch.randn(5, 128, device=dev).to(torch.bfloat16)
    x[1] = 0
    x[2, 77] = float("nan")
    x[3, 5] = float("inf")
    w = torch.ones(128, dtype=torch.bfloat16, device=dev)
    (q, s), _ = ops.rmsnorm_quantize(x, w, fmt=fmt)
    s = s.cpu().numpy()
    nan_byte = 0x7F if fmt == "nvfp4" else 0xFF
    assert not (unpacked(q, fmt)[1] & (0x7F if fmt == "mxfp8" else 7)).any() and not s[1].any()
    assert (s[2] == nan_byte).all()
    block = 5 // ops.QBLOCK[fmt]
    assert s[3, block] == nan_byte  # inf / inf; the rest of its row is finite / inf = 0
    for r in (0, 4):
        (q1, s1), _ = ops.rmsnorm_quantize(x[r:r + 1].clone(), w, fmt=fmt)
        assert torch.equal(q1[0], q[r]) and np.array_equal(s1.cpu().numpy()[0], s[r])


def test_norm_refusals():
    dev = device()
    x = torch.randn(2, 64, device=dev).to(torch.bfloat16)
    w = torch.ones(64, dtype=torch.bfloat16, device=dev)
    for bad in (lambda: ops.rmsnorm_quantize(x, w[:32]), lambda: ops.rmsnorm_quantize(x, w, fmt="int8"),
                lambda: ops.rmsnorm_quantize(x[:, :40], w[:40]), lambda: ops.rmsnorm_quantize(x, w, x.half()),
                lambda: ops.rmsnorm_quantize(x, w, residual_out=x.clone()),
                lambda: ops.rmsnorm_quantize(x, w, x, residual_out=x.float()),
                lambda: ops.rmsnorm_quantize(x, w, y=x.float()),
                lambda: ops.rmsnorm_quantize(x, w, tensor_scale=torch.ones(1, device=dev)),
                lambda: ops.silu_mul_quantize(x[:, :33]), lambda: ops.silu_mul_quantize(x, x[:1]),
                lambda: ops.silu_mul_quantize(x[:, :32].contiguous())):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(TypeError):
        ops.rmsnorm_quantize(x.float(), w)
    with pytest.raises(TypeError):
        ops.silu_mul_quantize(x.float())
    with pytest.raises(ops.MxStatusError, match="INVALID_ARG"):
        ops.rmsnorm_quantize(x, w, eps=-1.0)
    with pytest.raises(ops.MxStatusError, match="INVALID_ARG"):
        ops.rmsnorm_quantize(x, w, eps=float("nan"))
    k = 32768 + 32
    with pytest.raises(ops.MxStatusError, match="UNSUPPORTED"):
        ops.rmsnorm_quantize(torch.zeros(1, k, dtype=torch.bfloat16, device=dev),
                             torch.zeros(k, dtype=torch.bfloat16, device=dev))


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("M,K", [(1, 32), (3, 96), (129, 1056), (16, 14336), (700, 2080)])
def test_activation_against_fp64(fmt, M, K):
    dev = device()
    rng = np.random.default_rng(M + K)
    gb, gate = rand_bf16(rng, M, K, scale=4.0)
    gate = np.clip(gate, -30, 30)
    gb = bf16_bits_of(gate)
    ub, up = rand_bf16(rng, M, K)
    y = oracle.silu_mul(gate, up)
    both = bf16_to_dev(np.concatenate([gb, ub], axis=1), dev)
    g = scale_tensor(G[fmt], dev)
    q, s = ops.silu_mul_quantize(both, fmt=fmt, tensor_scale=g)
    check_quantised(unpacked(q, fmt), s.cpu().numpy(), y, fmt)
    q2, s2 = ops.silu_mul_quantize(bf16_to_dev(gb, dev), bf16_to_dev(ub, dev), fmt=fmt, tensor_scale=g)
    assert torch.equal(q, q2) and torch.equal(s, s2)
    pa = ops.silu_mul_quantize(both, fmt=fmt, tensor_scale=g, packed=True)
    rows, pad = packed_to_rows(pa, fmt)
    assert torch.equal(pa.x_q.view(M, -1), q) and np.array_equal(rows, s.cpu().numpy()) and not pad.any()


def test_activation_extremes():
    dev = device()
    gate = np.zeros((1, 64))
    gate[0, :6] = [-100.0, 100.0, -88.0, 88.5, -3e38, 3e38]
    gate[0, 32:] = -87.5  # a block of tiny values keeps its own scale
    up = np.ones((1, 64))
    bits = bf16_bits_of(np.concatenate([gate, up], axis=1))
    gate = synth.bf16_bits_to_f64(bits)[:, :64]
    q, s = ops.silu_mul_quantize(bf16_to_dev(bits, dev), fmt="mxfp8")
    y = oracle.silu_mul(gate, up)
    got = oracle.dequantize(q.cpu().numpy(), s.cpu().numpy())
    n = np.abs(y[:, :32]).max()
    assert np.abs(got[:, :32] - y[:, :32]).max() <= 2.0 ** -3 * n  # one block: 448 / 512 saturation at most
    assert (np.abs(got[:, 32:] - y[:, 32:]) <= 2.0 ** -3 * np.abs(y[:, 32:])).all()
    bits[0, 3] = bf16_bits_of(np.array([np.inf]))[0]
    q, s = ops.silu_mul_quantize(bf16_to_dev(bits, dev), fmt="mxfp8")
    assert s[0, 0] == 0xFF and s[0, 1] != 0xFF


def make_mlp(fmt, K, F, dev, seed=0):
    gen = torch.Generator(device="cpu").manual_seed(seed)
    mk = lambda *sh, std: (torch.randn(*sh, generator=gen) * std).to(torch.bfloat16).to(dev)  # noqa: E731
    w1, w2 = mk(2 * F, K, std=0.05), mk(K, F, std=0.05)
    nw = 1 + mk(K, std=0.1)
    deq = []
    packed = []
    for w in (w1, w2):
        if fmt == "mxfp8":
            q, s = ops.quantize(w)
            packed.append(ops.process_weights(q, s))
            deq.append(oracle.dequantize(q.cpu().numpy(), s.cpu().numpy()))
        else:
            g = None if fmt == "mxfp4" else (w.float().abs().amax() / 2688).reshape(1)
            q, s = ops.quantize_fp4(w, fmt, tensor_scale=g)
            packed.append(ops.process_weights_fp4(q, s, fmt, tensor_scale=g))
            deq.append(oracle.dequantize4(oracle.unpack(q.cpu().numpy()), s.cpu().numpy(), fmt,
                                          1.0 if g is None else float(g)))
    tx = None if fmt != "nvfp4" else torch.tensor([0.004], device=dev)
    th = None if fmt != "nvfp4" else torch.tensor([0.01], device=dev)
    return mlp.GatedMLP(nw, *packed, x_tensor_scale=tx, h_tensor_scale=th), nw, deq, tx, th


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("M", [1, 40, 300])
def test_mlp_block_is_its_steps_and_is_near_fp64(fmt, M):
    """The one call is bit-identical to the separate packed calls, and up to the order of fp32 sums to those with
    row-major scales; against fp64 the block differs by the 8- or 4-bit roundings that two fp32 paths take differently,
    which is rare: the rms of the difference stays under 1 % of the output's (bf16's own is 0.2 %)."""
    dev = device()
    K, F = 256, 640
    block, nw, (w1, w2), tx, th = make_mlp(fmt, K, F, dev)
    torch.manual_seed(M)
    x = torch.randn(M, K, device=dev).to(torch.bfloat16)
    res = (2 * torch.randn(M, K, device=dev)).to(torch.bfloat16)
    out, t = block(x, res)
    ops.check()
    gemm = ops.gemm_packed if fmt == "mxfp8" else ops.gemm_packed_fp4
    a, t2 = ops.rmsnorm_quantize(x, nw, res, fmt=fmt, tensor_scale=tx, packed=True)
    c = ops.silu_mul_quantize(gemm(a, block.gate_up), fmt=fmt, tensor_scale=th, packed=True)
    assert torch.equal(out, gemm(c, block.down)[0]) and torch.equal(t, t2)
    alone, none = block(x)
    assert none is None and alone.shape == x.shape
    (q, s), t2 = ops.rmsnorm_quantize(x, nw, res, fmt=fmt, tensor_scale=tx)
    lin = (lambda q, p, s, g: ops.linear(q, p, None, s)) if fmt == "mxfp8" else \
        (lambda q, p, s, g: ops.linear_fp4(q, p, None, s, tensor_scale=g))
    h = lin(q, block.gate_up, s, tx)
    q, s = ops.silu_mul_quantize(h, fmt=fmt, tensor_scale=th)
    steps = lin(q, block.down, s, th)
    assert torch.equal(t, t2) and out.shape == (M, K)
    # (the layers may split K differently between the two forms: fp32 order only)
    assert (out.float() - steps.float()).norm() <= 4e-3 * steps.float().norm()

    def fake(v, g):
        c, sc = oracle.quantize_any(v, fmt, 1.0 if g is None else float(g))
        return oracle.dequantize(c, sc) if fmt == "mxfp8" else oracle.dequantize4(c, sc, fmt, 1.0 if g is None else float(g))

    _, y = oracle.rmsnorm(x.double().cpu().numpy(), nw.double().cpu().numpy(), res.double().cpu().numpy())
    hh = to_bf16_f64(fake(y, tx) @ w1.T)
    ref = fake(oracle.silu_mul(hh[:, :F], hh[:, F:]), th) @ w2.T
    got = out.double().cpu().numpy()
    assert np.sqrt(np.mean((got - ref) ** 2)) <= 0.01 * np.sqrt(np.mean(ref ** 2))


def test_mlp_in_a_graph_and_refusals():
    dev = device()
    block, nw, _, tx, th = make_mlp("nvfp4", 256, 512, dev)
    x = torch.randn(2, 4, 256, device=dev).to(torch.bfloat16)
    res = torch.randn(2, 4, 256, device=dev)
    ref, t = block(x, res)
    assert ref.shape == x.shape and t.dtype == torch.float32
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, _ = block(x, res)
    out.zero_()
    graph.replay()
    assert torch.equal(out, ref)
    with pytest.raises(ValueError):
        mlp.GatedMLP(nw, block.down, block.gate_up)
    other, *_ = make_mlp("mxfp4", 256, 512, dev)
    with pytest.raises(ValueError):
        mlp.GatedMLP(nw, block.gate_up, other.down)
    for bad in (lambda: block(x[..., :128]), lambda: block(x, res[:1]), lambda: block(x, res.half()),
                lambda: ops.gated_mlp(x, nw[:128], block.gate_up, block.down),
                lambda: ops.gated_mlp(x, nw, block.down, block.gate_up),
                lambda: ops.gated_mlp(x, nw, other.gate_up, other.down, x_tensor_scale=tx)):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(ops.MxStatusError, match="workspace"):
        ops.gated_mlp(x, nw, block.gate_up, block.down, workspace=torch.empty(256, dtype=torch.uint8, device=dev))
    empty, t = block(x[:0], res[:0])
    assert empty.shape == (0, 4, 256) and t.shape == (0, 4, 256)


def banded(n_bytes, dev):
    """A buffer of n_bytes inside 4 KB bands of a known byte: (buffer, check that the bands are untouched)."""
    raw = torch.full((n_bytes + 8192,), 0xA5, dtype=torch.uint8, device=dev)
    return raw[4096:4096 + n_bytes], lambda: bool((raw[:4096] == 0xA5).all() and (raw[4096 + n_bytes:] == 0xA5).all())


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("packed", [0, 1])
@pytest.mark.parametrize("M,K", [(3, 96), (130, 1056)])
def test_every_call_writes_its_documented_bytes_only(fmt, packed, M, K):
    dev = device()
    lib, st = ops.load(), torch.cuda.current_stream().cuda_stream
    f = ops.QFMT[fmt]
    x = torch.randn(M, 2 * K, device=dev).to(torch.bfloat16)
    w = torch.randn(K, device=dev).to(torch.bfloat16)
    res = torch.randn(M, K, device=dev)
    qb = M * K // (1 if fmt == "mxfp8" else 2)
    sizes = ops.packed_sizes(1, M, K) if fmt == "mxfp8" else ops.packed_sizes_fp4(1, M, K, fmt)
    sb = sizes[1] if packed else M * K // ops.QBLOCK[fmt]
    ok = []

    def buf(n):
        b, check = banded(n, dev)
        ok.append(check)
        return b.data_ptr()

    assert lib.mxfp8_rmsnorm_quantize(f, x.data_ptr(), 2 * K, res.data_ptr(), K, 1, buf(4 * M * K), w.data_ptr(), 1e-6,
                                      None, M, K, buf(qb), buf(sb), packed, buf(2 * M * K), st) == 0
    assert lib.mxfp8_silu_mul_quantize(f, x.data_ptr(), 2 * K, x.data_ptr() + 2 * K, 2 * K, None, M, K, buf(qb), buf(sb),
                                       packed, st) == 0
    if fmt != "mxfp8":
        xd = x[:, :K].contiguous()
        if packed:
            assert lib.mxfp8_fp4_quantize_packed(f, xd.data_ptr(), 1, M, K, None, buf(qb), buf(sb), st) == 0
        else:
            assert lib.mxfp8_fp4_quantize(f, xd.data_ptr(), M, K, None, buf(qb), buf(sb), st) == 0
            q, s = ops.quantize_fp4(xd, fmt)
            assert lib.mxfp8_fp4_unpack(q.data_ptr(), M * K, buf(M * K), st) == 0
            assert lib.mxfp8_fp4_process_weights(f, q.data_ptr(), s.data_ptr(), 1, M, K, buf(qb), buf(sizes[1]), st) == 0
    torch.cuda.synchronize()
    assert all(check() for check in ok)


@pytest.mark.parametrize("fmt", FMTS)
def test_tensors_past_two_billion_elements(fmt):
    """Offsets beyond 32 bits: the last rows of a 2.2 G-element input come out as they do alone."""
    dev = device()
    M, K = 66000, 32768
    gen = torch.Generator(device=dev).manual_seed(1)
    x = torch.empty(M, K, dtype=torch.bfloat16, device=dev)
    x[:-4] = 1.0
    x[-4:] = torch.randn(4, K, device=dev, generator=gen).to(torch.bfloat16)
    w = torch.randn(K, device=dev, generator=gen).to(torch.bfloat16)
    (q, s), _ = ops.rmsnorm_quantize(x, w, fmt=fmt)
    (q1, s1), _ = ops.rmsnorm_quantize(x[-4:].clone(), w, fmt=fmt)
    assert torch.equal(q[-4:], q1) and torch.equal(s[-4:], s1)
    del q, s
    q, s = ops.silu_mul_quantize(x[:, :K // 2], x[:, K // 2:], fmt=fmt)
    q1, s1 = ops.silu_mul_quantize(x[-4:].clone(), fmt=fmt)
    assert torch.equal(q[-4:], q1) and torch.equal(s[-4:], s1)
    del q, s
    if fmt != "mxfp8":
        q, s = ops.quantize_fp4(x, fmt)
        q1, s1 = ops.quantize_fp4(x[-4:].clone(), fmt)
        assert torch.equal(q[-4:], q1) and torch.equal(s[-4:], s1)
        assert torch.equal(ops.unpack_fp4(q)[-4:].view(torch.uint8), ops.unpack_fp4(q1).view(torch.uint8))
