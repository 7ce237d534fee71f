"""A bias, or the weights' tensor scale, that the library's own kernel ahead in the stream has just written.

As in test_gpu_norm_weight_order.py: the products are let in before that kernel ends and must read the bias after it."""

import pytest
import torch

from _helpers import device
from mxfp8_block_scaled_02_gb300 import ops
from test_gpu_norm_weight_order import bf, check_order, producers

pytestmark = pytest.mark.gpu

# kernel -> (weights' format, M, N, K, path of ops.linear)
CASES = {
    "4-bit, tokens quantised inside": ("mxfp4", 4, 4096, 1024, None),
    "4-bit, few tokens": ("nvfp4", 40, 4096, 1024, None),
    "4-bit, one CTA a tile": ("mxfp4", 1, 14336, 512, None),
    "4-bit, two CTAs an SM": ("nvfp4", 3, 20000, 512, None),
    "4-bit, CTA pairs": ("nvfp4", 300, 4096, 512, None),
    "4-bit, K split in a cluster": ("mxfp4", 256, 4096, 14336, None),
    "4-bit, K split over pairs": ("mxfp4", 256, 1024, 28672, None),
    "MXFP8, few tokens": ("e4m3", 4, 4096, 1024, 1),
    "MXFP8, few tokens, one CTA a tile": ("e4m3", 4, 14336, 512, 1),
    "MXFP8, one CTA a tile": ("e4m3", 300, 1024, 512, 2),
    "MXFP8, CTA pairs": ("e4m3", 300, 4096, 512, 3),
    "MXFP8, K split over pairs": ("e4m3", 256, 2048, 4096, 0),
    "MXFP8, quantised inside": ("e4m3", 200, 512, 1024, 5),
}


def layer(gen, fmt, N, K):
    w = bf(gen, N, K, scale=0.02)
    return ops.process_weights(*ops.quantize(w)) if fmt == "e4m3" else ops.process_weights_fp4(*ops.quantize_fp4(w, fmt), fmt)


@pytest.mark.parametrize("name", CASES)
def test_bias_from_the_kernel_before(name):
    device()
    fmt, M, N, K, path = CASES[name]
    gen = torch.Generator(device="cuda").manual_seed(N + K)
    x, pw = bf(gen, M, K), layer(gen, fmt, N, K)
    for who, (writers, bias) in producers(N, gen).items():
        if fmt == "e4m3":
            check_order(writers, lambda: (ops.linear(x, pw, bias, path=path),), who)
        else:
            check_order(writers, lambda: (ops.linear_fp4(x, pw, bias),), who)


@pytest.mark.parametrize("M", [4, 40, 300])
def test_codes_with_a_bias_from_the_kernel_before(M):
    """The packed hand-over, where nothing stands between the bias's writer and the product."""
    device()
    gen = torch.Generator(device="cuda").manual_seed(M)
    N, K = 4096, 1024
    x = bf(gen, M, K)
    p4, p8 = layer(gen, "nvfp4", N, K), layer(gen, "e4m3", N, K)
    a4, a8 = ops.quantize_packed_fp4(x, 1, "nvfp4"), ops.quantize_packed(x)
    for who, (writers, bias) in producers(N, gen).items():
        check_order(writers, lambda: (ops.gemm_packed_fp4(a4, p4, bias),), who)
        check_order(writers, lambda: (ops.gemm_packed(a8, p8, bias),), who)


@pytest.mark.parametrize("M", [4, 40, 300])
def test_weight_tensor_scale_from_the_kernel_before(M):
    device()
    gen = torch.Generator(device="cuda").manual_seed(M)
    N, K, R = 4096, 1024, 256
    x, pw = bf(gen, M, K), layer(gen, "nvfp4", N, K)
    a = ops.quantize_packed_fp4(x, 1, "nvfp4")
    nw, zero = bf(gen, N), torch.zeros(R, N, device="cuda")
    t = torch.zeros(R, N, device="cuda")
    writers = [lambda v=v: ops.rmsnorm_quantize(v, nw, zero, residual_out=t)
               for v in (bf(gen, R, N).abs() + 0.5, bf(gen, R, N).abs() + 2.0)]
    pw.tensor_scale = t[R - 1, :1]
    check_order(writers, lambda: (ops.linear_fp4(x, pw),), "linear")
    check_order(writers, lambda: (ops.gemm_packed_fp4(a, pw),), "packed")
