"""The CTA-pair 4-bit product: every tile width, K split and ragged edge, exactly.

Codes with power-of-two scales make every product a multiple of 1/16 (1/64 after
the tensor scales 1/2) and sums of them far smaller than 2^24 of those, so fp32
adds them exactly in any order: the output must be the rounded exact value.
"""

import numpy as np
import pytest
import torch

import oracle
from _helpers import device, u8_to_dev
from mxfp8_block_scaled_02_gb300 import ops

pytestmark = pytest.mark.gpu
FMTS = ["mxfp4", "nvfp4"]

# (B, M, N, K): 128-column tiles; K split in a cluster of two pairs; K split
# with partials; 256-column tiles, one and several a pair
SHAPES = [(1, 300, 2040, 2080), (3, 500, 1000, 1056), (1, 512, 4096, 4096),
          (1, 500, 4000, 11264), (1, 500, 4000, 11296), (2, 260, 2056, 12320), (1, 300, 4096, 14336),
          (1, 200, 1016, 28704), (1, 250, 4000, 16416),
          (1, 1100, 4104, 544), (2, 1300, 4104, 1056)]


def operand(rng, fmt, B, R, K):
    codes = rng.integers(0, 16, size=(B, R, K), dtype=np.uint8)
    pick = rng.integers(0, 3, size=(B, R, K // ops.QBLOCK[fmt]))
    return codes, (126 + pick if fmt == "mxfp4" else 0x30 + 8 * pick).astype(np.uint8)


def exact_case(fmt, B, M, N, K):
    rng = np.random.default_rng(3 * B + 5 * M + 7 * N + K)
    x, w = operand(rng, fmt, B, M, K), operand(rng, fmt, B, N, K)
    g = 1.0 if fmt == "mxfp4" else 0.5
    bias = rng.integers(-64, 65, size=N).astype(np.float64)
    ref = torch.from_numpy(oracle.dequantize4(*x, fmt, g)) @ torch.from_numpy(oracle.dequantize4(*w, fmt, g)).mT
    ref = (ref + torch.from_numpy(bias)).float().to(torch.bfloat16)
    return x, w, g, bias, ref


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("B,M,N,K", SHAPES)
def test_exact_sums(fmt, B, M, N, K):
    dev = device()
    x, w, g, bias, ref = exact_case(fmt, B, M, N, K)
    sq = (lambda a: a) if B > 1 else (lambda a: a[0])
    gt = None if fmt == "mxfp4" else torch.tensor([g], dtype=torch.float32, device=dev)
    pw = ops.process_weights_fp4(u8_to_dev(sq(oracle.pack(w[0])), dev), u8_to_dev(sq(w[1]), dev), fmt, tensor_scale=gt)
    bt = torch.from_numpy(bias).to(torch.bfloat16).to(dev)
    xq, xs = u8_to_dev(sq(oracle.pack(x[0])), dev), u8_to_dev(sq(x[1]), dev)
    got = ops.linear_fp4(xq, pw, bt, xs, tensor_scale=gt)
    ops.check()
    assert torch.equal(got.cpu().view(ref.shape), ref)
    for _ in range(3):  # the same on every call, back to back on one stream
        again = ops.linear_fp4(xq, pw, bt, xs, tensor_scale=gt)
    ops.check()
    assert torch.equal(again, got)


@pytest.mark.parametrize("fmt", FMTS)
def test_nan_scales_stay_in_their_row(fmt):
    """A NaN block of x in the second half of K, where K is split in two."""
    dev = device()
    M, N, K = 300, 4096, 14336
    x, w, g, bias, ref = exact_case(fmt, 1, M, N, K)
    x[1][0, 170, -1] = 0xFF if fmt == "mxfp4" else 0x7F
    gt = None if fmt == "mxfp4" else torch.tensor([g], dtype=torch.float32, device=dev)
    pw = ops.process_weights_fp4(u8_to_dev(oracle.pack(w[0])[0], dev), u8_to_dev(w[1][0], dev), fmt, tensor_scale=gt)
    got = ops.linear_fp4(u8_to_dev(oracle.pack(x[0])[0], dev), pw, torch.from_numpy(bias).to(torch.bfloat16).to(dev),
                         u8_to_dev(x[1][0], dev), tensor_scale=gt)
    ops.check()
    got = got.cpu()
    assert got[170].isnan().all()
    keep = torch.arange(M) != 170
    assert torch.equal(got[keep], ref[0][keep])


def test_a_cluster_split_needs_no_workspace():
    assert ops.product_workspace_fp4(1, 512, 4096, 14336, "mxfp4") == 0
    assert ops.product_workspace_fp4(1, 250, 4000, 16416, "mxfp4") > 0
