"""A norm weight that the library's own kernel ahead in the stream has just written (an adaptive norm's, for one).

Those kernels let the next one start before they end; the norm must read its weight after they have.  The buffer that
holds the weight gets another content from call to call, so that an early read finds the content before."""

import pytest
import torch

from _helpers import device
from mxfp8_block_scaled_02_gb300 import mlp, ops

pytestmark = pytest.mark.gpu


def bf(gen, *shape, scale=1.0):
    return (torch.randn(*shape, device="cuda", generator=gen) * scale).bfloat16()


def producers(n, gen):
    """name -> (two writers, the bf16 [n] view they write): each way a kernel that triggers early leaves a bf16 row."""
    K, R = 14336, 256
    made = {}
    w = bf(gen, n, K, scale=0.02)
    for name, pack, linear in (("4-bit linear", lambda: ops.process_weights_fp4(*ops.quantize_fp4(w, "nvfp4"), "nvfp4"),
                                ops.linear_fp4),
                               ("MXFP8 linear", lambda: ops.process_weights(*ops.quantize(w)), ops.linear)):
        pw, out = pack(), torch.zeros(1, n, dtype=torch.bfloat16, device="cuda")
        xs = [bf(gen, 1, K), bf(gen, 1, K)]
        made[name] = ([lambda x=x, pw=pw, out=out, linear=linear: linear(x, pw, out=out) for x in xs], out[0])
    nw, xs = bf(gen, n), [bf(gen, R, n), bf(gen, R, n)]
    y, t = (torch.zeros(R, n, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    made["norm's y"] = ([lambda x=x: ops.rmsnorm_quantize(x, nw, y=y) for x in xs], y[R - 1])
    made["norm's sum"] = ([lambda x=x: ops.rmsnorm_quantize(x, nw, xs[0], residual_out=t) for x in xs], t[R - 1])
    return made


def bytes_of(res):
    return [t.clone().contiguous().view(torch.uint8) for t in res]


def check_order(writers, consumer, what):
    """consumer() after each writer, in a row and in a graph, gives what it gives after a synchronisation."""
    refs = []
    for write in writers:
        write()
        torch.cuda.synchronize()
        refs.append(bytes_of(consumer()))
        torch.cuda.synchronize()
    assert any(not torch.equal(a, b) for a, b in zip(*refs)), what  # the content matters

    def in_a_row():
        got = []
        for _ in range(4):
            for i, write in enumerate(writers):
                write()
                got.append((i, consumer()))
        return got

    got = in_a_row()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = in_a_row()
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    ops.check()
    for i, res in got + captured:
        assert all(torch.equal(a, b) for a, b in zip(bytes_of(res), refs[i])), what


@pytest.mark.parametrize("n", [4096, 8192, 12288])
def test_norm_weight_from_the_kernel_before(n):
    device()
    gen = torch.Generator(device="cuda").manual_seed(n)
    x, res = bf(gen, 4, n), bf(gen, 4, n)

    def norm(w, r):
        (q, s), t = ops.rmsnorm_quantize(x, w, r)
        return (q, s)

    for name, (writers, w) in producers(n, gen).items():
        check_order(writers, lambda: norm(w, None), f"{name}, no residual")
        check_order(writers, lambda: norm(w, res), f"{name}, residual")


def test_mlp_norm_weight_from_the_kernel_before():
    device()
    gen = torch.Generator(device="cuda").manual_seed(1)
    n, f = 1024, 1024
    pack = lambda w: ops.process_weights_fp4(*ops.quantize_fp4(w, "mxfp4"), "mxfp4")  # noqa: E731
    up, down = pack(bf(gen, 2 * f, n, scale=0.03)), pack(bf(gen, n, f, scale=0.03))
    x = bf(gen, 3, n)
    for name, (writers, w) in producers(n, gen).items():
        block = mlp.GatedMLP(w, up, down)
        check_order(writers, lambda: (block(x)[0],), name)
