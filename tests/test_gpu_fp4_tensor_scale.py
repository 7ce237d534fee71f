"""NVFP4 with tensor scales g of every size: the rule s = E4M3(amax / (6 g)) holds for every g >= 0, also where 6 g or
its inverse leaves the normal fp32 range, and a block of zeros has the scale 0 whatever g is."""

import numpy as np
import pytest
import torch

import oracle
from _helpers import bf16_to_dev, device
from mxfp8_block_scaled_02_gb300 import ops, synth
from test_gpu_fp4 import atoms_of, bf16_bits_of, rand_bf16, scale_tensor

pytestmark = pytest.mark.gpu

LIM = 2.0 ** -126 / 6
# zero (the amax of an all-zero tensor), subnormal, 6 g around 2^-128 and 2^-126, ordinary, 6 g around 2^126 and 2^128
SCALES = [0.0, 1e-45, 1e-40, LIM / 4 * 0.999, LIM / 4 * 1.001, LIM * 0.7, LIM * 0.9999, LIM, LIM * 1.0001, 1e-30, 1.0,
          1e37, 2.0 ** 126 / 6 * 0.9999, 2.0 ** 126 / 6 * 1.0001, 5e37, 6e37]


def blocks_for(g, rng):
    """bf16 [4, 512]: zero blocks, blocks whose quotient amax / (6 g) lies all over E4M3's range and on its rounding
    boundaries (as near as bf16 comes), tiny and huge blocks, an Inf and a NaN block."""
    rows = [np.zeros(512)]
    with np.errstate(over="ignore"):
        six_g = float(np.float32(6) * np.float32(g)) or 1.0
    quotients = np.concatenate([[2.0 ** -11, 2.0 ** -10, 1.5 * 2.0 ** -9, 1.0, 17 / 16, 19 / 16, 447.0, 448.0, 464.0, 1e4],
                                np.exp2(rng.uniform(-12, 10, 22))])
    amax = np.minimum(quotients * six_g, 3.3e38)
    rows.append((amax[:, None] * rng.uniform(-1, 1, (32, 16))).ravel())
    rows[-1][::16] = amax
    mixed = np.zeros((32, 16))
    mixed[1::4] = amax[1::4, None]
    mixed[2] = 9.2e-41
    mixed[3] = -3.3e38
    mixed[4, 5], mixed[8, 7] = np.inf, np.nan
    rows.append(mixed.ravel())
    rows.append(rng.standard_normal(512))
    with np.errstate(over="ignore"):
        return bf16_bits_of(np.stack(rows))


@pytest.mark.parametrize("g", SCALES)
def test_scale_bytes_and_codes_follow_the_rule(g):
    dev = device()
    g = float(np.float32(g))
    bits = blocks_for(g, np.random.default_rng(7))
    codes, s = oracle.quantize4(synth.bf16_bits_to_f64(bits), "nvfp4", g)
    assert not s[0].any() and (s[2, 4] == 0x7F) and (s[2, 8] == 0x7F)
    xt, gt = bf16_to_dev(bits, dev), scale_tensor(g, dev)
    q_d, s_d = ops.quantize_fp4(xt, "nvfp4", tensor_scale=gt)
    assert np.array_equal(s_d.cpu().numpy(), s)
    assert np.array_equal(q_d.cpu().numpy(), oracle.pack(codes))
    pa = ops.quantize_packed_fp4(xt, 1, "nvfp4", tensor_scale=gt)
    want, mask = atoms_of(s, 512, "nvfp4")
    assert np.array_equal(pa.x_q.cpu().numpy().reshape(4, -1), oracle.pack(codes))
    assert np.array_equal(pa.sf_packed.cpu().numpy()[mask], want[mask])


def check_rounding_of(q_d, s_d, y, g):
    """The bytes are those that y (1 - d), y or y (1 + d) rounds to, d = 1e-5 the fp32 error of y (as derived in
    test_gpu_fused_steps.py)."""
    got_s, got = s_d.cpu().numpy(), oracle.unpack(q_d.cpu().numpy())
    ok_s, ok = np.zeros(got_s.shape, bool), np.zeros(got.shape, bool)
    for f in (1 - 1e-5, 1.0, 1 + 1e-5):
        c, s = oracle.quantize4(y * f, "nvfp4", g)
        ok_s |= s == got_s
        ok |= np.repeat(s == got_s, 16, axis=-1) & ((c == got) | ((c & 7) + (got & 7) == 0))
    assert ok_s.all() and ok.all()


@pytest.mark.parametrize("g", [0.0, 1e-45, 1e-40, LIM * 0.7, 5e37])
def test_norm_and_activation_follow_it_too(g):
    """A zero row stays zero; the others' blocks have magnitudes all over fp32's range."""
    dev = device()
    g = float(np.float32(g))
    rng = np.random.default_rng(8)
    gt = scale_tensor(g, dev)
    xb, x = rand_bf16(rng, 3, 512)
    w = np.exp2(rng.integers(-126, 20, 32)).repeat(16)
    xb[1], x[1] = 0, 0.0
    (q_d, s_d), _ = ops.rmsnorm_quantize(bf16_to_dev(xb, dev), bf16_to_dev(bf16_bits_of(w), dev), eps=1e-6, fmt="nvfp4",
                                         tensor_scale=gt)
    assert not s_d[1].any() and not (q_d[1] & 0x77).any()
    check_rounding_of(q_d, s_d, oracle.rmsnorm(x, w, None, 1e-6)[1], g)
    gate = rng.uniform(1.0, 30.0, (3, 512))
    up = np.where(np.arange(3)[:, None] == 1, 0.0, x * w)
    both = bf16_bits_of(np.concatenate([gate, up], axis=1))
    q_d, s_d = ops.silu_mul_quantize(bf16_to_dev(both, dev), fmt="nvfp4", tensor_scale=gt)
    assert not s_d[1].any() and not (q_d[1] & 0x77).any()
    both = synth.bf16_bits_to_f64(both)
    check_rounding_of(q_d, s_d, oracle.silu_mul(both[:, :512], both[:, 512:]), g)


@pytest.mark.parametrize("g", [0.0, 1e-45, 1e-40])
@pytest.mark.parametrize("M", [1, 8, 40, 300])
def test_a_zero_tensor_gives_the_bias(g, M):
    """x all zero, calibrated to g = amax / 2688 = 0 or to next to nothing; zero weights with such a scale likewise."""
    dev = device()
    rng = np.random.default_rng(M)
    N, K = 264, 544
    gt = scale_tensor(float(np.float32(g)), dev)
    w = bf16_to_dev(rand_bf16(rng, N, K)[0], dev)
    bias = bf16_to_dev(rand_bf16(rng, N)[0], dev)
    zero = torch.zeros(M, K, dtype=torch.bfloat16, device=dev)
    pw = ops.process_weights_fp4(*ops.quantize_fp4(w, "nvfp4"), "nvfp4")
    out = ops.linear_fp4(zero, pw, bias, tensor_scale=gt)
    assert torch.equal(out, bias.expand(M, N))
    pa = ops.quantize_packed_fp4(zero, 1, "nvfp4", tensor_scale=gt)
    assert torch.equal(ops.gemm_packed_fp4(pa, pw, bias)[0], out)
    none = ops.process_weights_fp4(*ops.quantize_fp4(torch.zeros_like(w), "nvfp4", tensor_scale=gt), "nvfp4", tensor_scale=gt)
    x = bf16_to_dev(rand_bf16(rng, M, K)[0], dev)
    assert torch.equal(ops.linear_fp4(x, none, bias), out)
    ops.check()


@pytest.mark.parametrize("M", [1, 5, 8])
@pytest.mark.parametrize("g", [1e-45, 1e-40, LIM * 0.7, 5e37])
def test_few_tokens_quantised_inside_give_the_same_bytes(g, M):
    dev = device()
    rng = np.random.default_rng(M)
    N, K = 264, 512
    g = float(np.float32(g))
    bits = blocks_for(g, rng)
    bits = np.resize(bits[[1, 0, 3]], (M, K))
    xt, gt = bf16_to_dev(bits, dev), scale_tensor(g, dev)
    pw = ops.process_weights_fp4(*ops.quantize_fp4(bf16_to_dev(rand_bf16(rng, N, K)[0], dev), "nvfp4"), "nvfp4")
    q, s = ops.quantize_fp4(xt, "nvfp4", tensor_scale=gt)
    assert np.array_equal(s.cpu().numpy(), oracle.quantize4(synth.bf16_bits_to_f64(bits), "nvfp4", g)[1])
    codes = ops.linear_fp4(q, pw, x_scale=s, tensor_scale=gt)
    inside = ops.linear_fp4(xt, pw, tensor_scale=gt)
    ops.check()
    assert torch.equal(inside.view(torch.int16), codes.view(torch.int16)) and not torch.isnan(inside).any()
