"""Routing of more tokens than 64 a CTA: several groups one after the other in every CTA."""

import numpy as np
import pytest
import torch

import oracle
from _grouped import bf16_round, pack, to_bf16, to_dev, weights
from _helpers import device
from mxfp8_block_scaled_02_gb300 import mlp, ops
from test_gpu_route import assert_routing, restated_steps

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T,E,k", [(10241, 64, 8), (10241, 512, 4), (16384, 256, 4), (30000, 64, 8), (20481, 512, 2)])
def test_route_again_and_again(T, E, k):
    dev = device()
    z = np.random.default_rng(T + E).standard_normal((T, E)).astype(np.float32) * 3
    z[T // 2] = -np.inf
    zd = to_dev(z, dev)
    r = ops.route(zd, k, renormalize=True)
    want = oracle.route(z.astype(np.float64), k, "softmax", True)
    assert_routing(r, want, z)
    for _ in range(100):
        again = ops.route(zd, k, renormalize=True)
        for name in ("ids", "weights", "offsets", "rows", "positions"):
            assert torch.equal(getattr(again, name), getattr(r, name)), name


@pytest.mark.parametrize("fmt", ["mxfp8", "fp8_128"])
def test_expert_mlp_of_a_long_prompt(fmt):
    dev = device()
    rng = np.random.default_rng(1)
    T, E, k, K, F = 12000, 64, 4, 256, 128
    q1, s1, _ = weights(rng, fmt, E, 2 * F, K)
    q2, s2, _ = weights(rng, fmt, E, K, F)
    p1, p2 = pack(ops, q1, s1, fmt, dev), pack(ops, q2, s2, fmt, dev)
    x, z = to_bf16(bf16_round(rng.standard_normal((T, K))), dev), rng.standard_normal((T, E)).astype(np.float32)
    want = oracle.route(z.astype(np.float64), k, "softmax", True)
    z = to_dev(z, dev)
    r = ops.route(z, k, renormalize=True)
    assert np.array_equal(r.rows.cpu().numpy(), want["rows"]) and np.array_equal(r.positions.cpu().numpy(), want["positions"])
    block = mlp.ExpertMLP(p1, p2, k, renormalize=True)
    out = block(x, z)
    ops.check()
    assert torch.equal(out, restated_steps(x, z, p1, p2, k, None, renormalize=True))
    for _ in range(20):
        assert torch.equal(block(x, z), out)
