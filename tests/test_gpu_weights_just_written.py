"""Weights that an ordinary kernel has written directly before the product that reads them.

The block-128 product loads its first weights without waiting for the kernel ahead in the stream, which
is right because that kernel's dependents start when it has finished: the calls that make weights, and
copies, do not let them start early."""

import numpy as np
import pytest
import torch

from _grouped import bf16_round, to_bf16
from _helpers import device
from mxfp8_block_scaled_02_gb300 import ops

pytestmark = pytest.mark.gpu

# rows of x, N, K: quantised inside the product, quantised before it, a K split, CTA pairs
SHAPES = [(1, 4096, 1024), (8, 1032, 400), (24, 2056, 1040), (40, 20488, 272), (515, 4104, 400)]


@pytest.mark.parametrize("how", ["quantised", "copied", "quantised, a call between"])
@pytest.mark.parametrize("codes", [False, True])
@pytest.mark.parametrize("M,N,K", SHAPES)
def test_weights_just_written(M, N, K, codes, how):
    dev = device()
    rng = np.random.default_rng(M + N)
    x = to_bf16(bf16_round(rng.standard_normal((M, K))), dev)
    xq, xs = ops.quantize_fp8_128(x)
    z = torch.randn(16, 8, device=dev)
    ws = [to_bf16(bf16_round(rng.standard_normal((N, K))), dev) for _ in range(3)]
    made = [ops.process_weights_fp8_128(*ops.quantize_weights_fp8_128(w)) for w in ws]

    def product(pw):
        return ops.linear_fp8_128(xq, pw, x_scale=xs) if codes else ops.linear_fp8_128(x, pw)

    want = [product(pw) for pw in made]
    kept = ops.process_weights_fp8_128(made[0].w_packed.view(N, K).clone(), made[0].sf_packed.view(torch.float32).clone()
                                       .view(-(-N // 128), -(-K // 128)))
    torch.cuda.synchronize()
    got = []
    for i in range(60):
        if how == "copied":  # new weights in place, codes last or scales last
            for t in ("w_packed", "sf_packed") if i & 1 else ("sf_packed", "w_packed"):
                getattr(kept, t).copy_(getattr(made[i % 3], t))
            got.append(product(kept))
        else:
            pw = ops.process_weights_fp8_128(*ops.quantize_weights_fp8_128(ws[i % 3]))
            if how == "quantised":
                got.append(product(pw))
            else:  # a kernel that lets the product start before it has waited itself
                ops.route(z, 2)
                got.append(product(pw))
    torch.cuda.synchronize()
    ops.check()
    assert all(torch.equal(y, want[i % 3]) for i, y in enumerate(got))
