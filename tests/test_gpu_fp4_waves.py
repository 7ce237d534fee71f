"""The few-token 4-bit product with more weight tiles than SMs (two CTAs an SM)."""

import numpy as np
import pytest
import torch

import oracle
from _helpers import device, u8_to_dev
from mxfp8_block_scaled_02_gb300 import ops

pytestmark = pytest.mark.gpu
FMTS = ["mxfp4", "nvfp4"]


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("B,M,N,K", [(1, 1, 20008, 1056), (1, 5, 24000, 4128), (1, 30, 20008, 2080), (1, 64, 19600, 1312),
                                     (1, 100, 20008, 2080), (1, 128, 30000, 544), (16, 20, 1600, 1056), (2, 16, 16384, 32)])
def test_exact_sums(fmt, B, M, N, K):
    """Codes with power-of-two scales: fp32 adds every product exactly, so the output is the rounded exact value."""
    dev = device()
    rng = np.random.default_rng(B + 3 * M + 5 * N + 7 * K)
    sq = (lambda a: a) if B > 1 else (lambda a: a[0])

    def operand(R):
        pick = rng.integers(0, 3, size=(B, R, K // ops.QBLOCK[fmt]))
        return (rng.integers(0, 16, size=(B, R, K), dtype=np.uint8),
                (126 + pick if fmt == "mxfp4" else 0x30 + 8 * pick).astype(np.uint8))

    x, w = operand(M), operand(N)
    bias = rng.integers(-64, 65, size=N).astype(np.float64)
    ref = torch.from_numpy(oracle.dequantize4(*x, fmt)) @ torch.from_numpy(oracle.dequantize4(*w, fmt)).mT
    ref = (ref + torch.from_numpy(bias)).float().to(torch.bfloat16)
    pw = ops.process_weights_fp4(u8_to_dev(sq(oracle.pack(w[0])), dev), u8_to_dev(sq(w[1]), dev), fmt)
    bt = torch.from_numpy(bias).to(torch.bfloat16).to(dev)
    for _ in range(2):
        got = ops.linear_fp4(u8_to_dev(sq(oracle.pack(x[0])), dev), pw, bt, u8_to_dev(sq(x[1]), dev))
        ops.check()
        assert torch.equal(got.cpu().view(ref.shape), ref)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("M,N,K", [(1, 20008, 4128), (2, 24000, 4096), (2, 20008, 8224), (4, 20000, 1024), (16, 20008, 512)])
def test_bf16_tokens_give_the_bytes_of_the_quantise_call(fmt, M, N, K):
    """One or two tokens, or a short K, are quantised in the product's kernel, with rings of every fill."""
    dev = device()
    gen = torch.Generator(device=dev).manual_seed(M + N + K)
    x = torch.randn(M, K, device=dev, generator=gen).bfloat16()
    w = (torch.randn(N, K, device=dev, generator=gen) * 0.02).bfloat16()
    g = None if fmt == "mxfp4" else torch.tensor([0.01], device=dev)
    pw = ops.process_weights_fp4(*ops.quantize_fp4(w, fmt), fmt)
    q, s = ops.quantize_fp4(x, fmt, tensor_scale=g)
    codes = ops.linear_fp4(q, pw, x_scale=s, tensor_scale=g)
    for _ in range(3):
        assert torch.equal(ops.linear_fp4(x, pw, tensor_scale=g), codes)
    ops.check()
