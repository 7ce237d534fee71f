"""bf16 tokens quantised inside the few-token 4-bit product: up to eight rows, several tasks of two rows a stage, rings
that are refilled, one and two CTAs an SM.  The output is bit for bit that of the codes the quantise call gives.

A call quantises inside exactly when its workspace is empty, so each case says which side of the rule it is on."""

import pytest
import torch

from _helpers import device
from mxfp8_block_scaled_02_gb300 import ops

pytestmark = pytest.mark.gpu
FMTS = ["mxfp4", "nvfp4"]
# (N, K): K split over 8, 4 and 2 CTAs of 7, 14 and 28 stages and one CTA of 56 (rings hold 9 or 10); ragged N and K; two
# CTAs an SM (rings of 5) with 2, 17 and 33 stages
SHAPES = [(1000, 14336), (4096, 14336), (8192, 14336), (14336, 14336), (520, 4128), (8200, 8224), (20008, 512),
          (20008, 4128), (24000, 8224)]


def inputs(M, N, K, fmt, dev):
    gen = torch.Generator(device=dev).manual_seed(M + 3 * N + 7 * K)
    x = torch.randn(M, K, device=dev, generator=gen)
    x *= torch.exp2(torch.randint(-8, 9, (M, K // 32), device=dev, generator=gen).float()).repeat_interleave(32, 1)
    x[M // 2, :32] = 0.0
    w = (torch.randn(N, K, device=dev, generator=gen) * 0.02).bfloat16()
    bias = torch.randn(N, device=dev, generator=gen).bfloat16()
    g = None if fmt == "mxfp4" else torch.tensor([0.37], device=dev)
    return x.bfloat16(), ops.process_weights_fp4(*ops.quantize_fp4(w, fmt), fmt), bias, g


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("N,K", SHAPES)
def test_every_row_count_up_to_the_rules_edge(fmt, N, K):
    dev = device()
    for M in (1, 2, 3, 4, 5, 6, 7, 8, 9):
        x, pw, bias, g = inputs(M, N, K, fmt, dev)
        assert (ops.workspace_size_fp4(1, M, N, K, False, fmt) == 0) == (M <= 8)
        q, s = ops.quantize_fp4(x, fmt, tensor_scale=g)
        codes = ops.linear_fp4(q, pw, bias, s, tensor_scale=g)
        for _ in range(3):
            assert torch.equal(ops.linear_fp4(x, pw, bias, tensor_scale=g), codes), (M, N, K)
        ops.check()


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("M", [3, 6, 8])
@pytest.mark.parametrize("N,K", [(4096, 14336), (20008, 4128)])
def test_nonfinite_tokens_stay_in_their_row(fmt, M, N, K):
    dev = device()
    x, pw, bias, g = inputs(M, N, K, fmt, dev)
    x[0, K - 1], x[M - 1, 5] = float("inf"), float("nan")
    got = ops.linear_fp4(x, pw, bias, tensor_scale=g)
    q, s = ops.quantize_fp4(x, fmt, tensor_scale=g)
    codes = ops.linear_fp4(q, pw, bias, s, tensor_scale=g)
    ops.check()
    assert torch.equal(got.view(torch.int16), codes.view(torch.int16))
    assert torch.isnan(got[0]).all() and torch.isnan(got[M - 1]).all() and torch.isfinite(got[1:M - 1]).all()


@pytest.mark.parametrize("fmt", FMTS)
def test_eight_tokens_back_to_back_in_a_graph(fmt):
    """Layer after layer, each reading the one before: every launch starts while its predecessor still runs."""
    dev = device()
    _, up, bias_up, g = inputs(8, 14336, 4096, fmt, dev)
    x, down, bias, _ = inputs(8, 4096, 14336, fmt, dev)
    x = x[:, :4096].contiguous()

    def chain():
        h = x
        for _ in range(4):
            h = ops.linear_fp4(ops.linear_fp4(h, up, bias_up, tensor_scale=g), down, bias, tensor_scale=g)
        return h

    def steps():
        h = x
        for _ in range(4):
            for pw, b in ((up, bias_up), (down, bias)):
                q, s = ops.quantize_fp4(h, fmt, tensor_scale=g)
                torch.cuda.synchronize()
                h = ops.linear_fp4(q, pw, b, s, tensor_scale=g)
                torch.cuda.synchronize()
        return h

    ref = steps()
    assert torch.equal(chain(), ref)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = chain()
    for _ in range(3):
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, ref)
    ops.check()
