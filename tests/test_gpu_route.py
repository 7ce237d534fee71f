"""Expert routing, the weighted sum, and the mixture-of-experts MLP."""

import numpy as np
import pytest
import torch

import oracle
from _grouped import bf16_round, f64, fake, pack, to_bf16, to_dev, weights
from _helpers import device
from mxfp8_block_scaled_02_gb300 import mlp, ops

pytestmark = pytest.mark.gpu


def assert_routing(r: ops.Routing, want: dict, z: np.ndarray, scale: float = 1.0) -> None:
    for name in ("ids", "offsets", "rows", "positions"):
        assert np.array_equal(getattr(r, name).cpu().numpy(), want[name]), name
    # exp within 2 ulp of an argument that is off by half an ulp of |z - top| <= 2^7: 2^-17 at the
    # most, and as much again for the sum's terms; sums of up to 512 terms and the divisions 2^-15
    w = f64(r.weights)
    span = np.abs(np.where(np.isfinite(z), z, 0)).max() + 1
    rel = 4 * (span * 2.0 ** -24 + 2 * 2.0 ** -23) + 600 * 2.0 ** -24
    assert (np.abs(w - want["weights"]) <= rel * np.abs(want["weights"]) + 2.0 ** -126 * abs(scale)).all()


SIZES = [(1, 1, 1), (1, 8, 8), (3, 5, 2), (16, 64, 8), (32, 64, 8), (33, 64, 8), (64, 33, 4), (65, 128, 6), (1281, 40, 3),
         (200, 256, 8), (1000, 512, 32), (130, 100, 1),
         (20000, 16, 2)]


@pytest.mark.parametrize("T,E,k", SIZES)
@pytest.mark.parametrize("scoring,renormalize,scale", [("softmax", False, 1.0), ("softmax", True, 2.5), ("sigmoid", True, 1.0)])
def test_route(T, E, k, scoring, renormalize, scale):
    dev = device()
    z = np.random.default_rng(T + E).standard_normal((T, E)).astype(np.float32) * 3
    r = ops.route(to_dev(z, dev), k, scoring=scoring, renormalize=renormalize, scale=scale)
    assert_routing(r, oracle.route(z.astype(np.float64), k, scoring, renormalize, scale), z, scale)


@pytest.mark.parametrize("T", [7, 64, 300])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_ties_masks_and_strides(T, dtype):
    """Equal logits, -inf and NaN, tokens with fewer than k experts or none, all on one expert; rows of a wider tensor."""
    dev = device()
    rng = np.random.default_rng(T)
    E, k = 40, 6
    z = rng.integers(-3, 4, (T, E)).astype(np.float64)
    z[0] = -np.inf
    z[1] = np.nan
    z[2, 3:] = -np.inf
    z[3, ::2] = np.nan
    z[4] = -0.0
    z[4, 5] = 0.0
    z[5] = -80.0
    z[6] = 3e38
    z[7:20, 9] = 50.0
    z = f64(torch.from_numpy(z).to(dtype))
    wide = torch.full((T, E + 24), 99.0, dtype=dtype, device=dev)
    wide[:, 3:3 + E] = torch.from_numpy(z).to(dtype).to(dev)
    view = wide[:, 3:3 + E]
    for scoring in ("softmax", "sigmoid"):
        want = oracle.route(z, k, scoring, True)
        assert (want["ids"] == -1).any()
        assert_routing(ops.route(view, k, scoring=scoring, renormalize=True), want, np.zeros(1))
    t = view.t().contiguous().t()  # columns contiguous: copied
    assert torch.equal(ops.route(t, k).ids, ops.route(view, k).ids)


def test_weights_that_underflow_stay_zero():
    dev = device()
    r = ops.route(torch.full((2, 8), -1e30, device=dev), 3, scoring="sigmoid", renormalize=True)
    assert r.ids.tolist() == [[0, 1, 2]] * 2 and (r.weights == 0).all()


def test_all_tokens_on_one_expert_and_none():
    dev = device()
    z = np.full((500, 12), -np.inf, dtype=np.float32)
    z[:, 7] = 1.0
    r = ops.route(to_dev(z, dev), 3)
    assert r.offsets.tolist() == [0] * 8 + [500] * 5
    assert r.rows.tolist() == list(range(500)) + [-1] * 1000
    empty = ops.route(torch.empty(0, 12, device=dev), 3)
    assert empty.offsets.tolist() == [0] * 13 and tuple(empty.ids.shape) == (0, 3)


@pytest.mark.parametrize("T", [50, 5000])
def test_route_again_and_in_a_graph(T):
    """Nothing depends on the order of atomics: repeated calls give the same, and a graph follows the logits."""
    dev = device()
    g = torch.Generator(device="cuda").manual_seed(0)
    zs = [torch.randn(T, 64, device=dev, generator=g) for _ in range(3)]
    want = [ops.route(z, 8) for z in zs]
    z = zs[0].clone()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        r = ops.route(z, 8)
    for i in (1, 2, 0, 1):
        z.copy_(zs[i])
        graph.replay()
        again = ops.route(zs[i], 8)
        for name in ("ids", "weights", "offsets", "rows", "positions"):
            assert torch.equal(getattr(r, name), getattr(want[i], name)), name
            assert torch.equal(getattr(again, name), getattr(want[i], name)), name


@pytest.mark.parametrize("T,k,N,R", [(1, 1, 8, 1), (5, 3, 264, 15), (70, 8, 1000, 560), (33, 32, 520, 900)])
@pytest.mark.parametrize("with_add", [False, True])
def test_combine(T, k, N, R, with_add):
    """A sum of k products and add in fp32 ((k + 1) 2^-24 of the terms' magnitudes), rounded once (2^-8)."""
    dev = device()
    rng = np.random.default_rng(T * k)
    y = bf16_round(rng.standard_normal((R, N)))
    pos = rng.integers(-1, R + 1, (T, k)).astype(np.int32)
    pos[0] = -1  # a token without experts
    w = rng.random((T, k)).astype(np.float32)
    add = bf16_round(rng.standard_normal((T, N))) if with_add else None
    routing = ops.Routing(None, to_dev(w, dev), None, None, to_dev(pos, dev))
    add_d = None
    if with_add:  # rows of a wider tensor
        add_d = torch.zeros(T, N + 16, dtype=torch.bfloat16, device=dev)
        add_d[:, 8:8 + N] = to_bf16(add, dev)
        add_d = add_d[:, 8:8 + N]
    out = ops.combine(to_bf16(y, dev), routing, add=add_d)
    ref = oracle.combine(y, pos, w, add)
    mag = oracle.combine(np.abs(y), pos, w, None if add is None else np.abs(add))
    assert (np.abs(f64(out) - ref) <= 2.0 ** -8 * np.abs(ref) + (k + 1) * 2.0 ** -23 * mag).all()


def restated_steps(x, logits, gate_up, down, k, add, **how):
    """The block by its public calls."""
    r = ops.route(logits, k, **how)
    h = ops.grouped_linear(x, gate_up, r.offsets, rows=r.rows)
    fmt = "fp8_128" if gate_up.fmt == "fp8_128" else "mxfp8"
    cq, cs = ops.silu_mul_quantize(h, fmt=fmt)
    y = ops.grouped_linear(cq, down, r.offsets, cs)
    return ops.combine(y, r, add=add)


@pytest.mark.parametrize("fmt", ["mxfp8", "fp8_128"])
@pytest.mark.parametrize("T,E,k,K,F", [(1, 8, 2, 256, 128), (5, 16, 4, 384, 256), (70, 8, 8, 256, 384), (600, 4, 2, 512, 256),
                                       (3000, 4, 2, 256, 384), (2500, 9, 4, 512, 128), (1700, 3, 1, 640, 400)])
def test_expert_mlp_is_its_steps(fmt, T, E, k, K, F):
    """Bit for bit the calls it is made of, and near the fp64 block."""
    if fmt == "mxfp8" and F % 128:
        pytest.skip("K is a multiple of 128 in MXFP8")
    dev = device()
    rng = np.random.default_rng(T + F)
    q1, s1, w1 = weights(rng, fmt, E, 2 * F, K)
    q2, s2, w2 = weights(rng, fmt, E, K, F)
    p1, p2 = pack(ops, q1, s1, fmt, dev), pack(ops, q2, s2, fmt, dev)
    x, z = bf16_round(rng.standard_normal((T, K))), rng.standard_normal((T, E)).astype(np.float32)
    if T > 4:
        z[2] = -np.inf  # a padded token
        z[3, 1:] = -np.inf
    add = bf16_round(rng.standard_normal((T, K)))
    xd, zd, ad = to_bf16(x, dev), to_dev(z, dev), to_bf16(add, dev)
    block = mlp.ExpertMLP(p1, p2, k, renormalize=True, scale=1.5)
    out = block(xd, zd, add=ad)
    ops.check()
    assert torch.equal(out, restated_steps(xd, zd, p1, p2, k, ad, renormalize=True, scale=1.5))
    assert torch.equal(out, block(xd, zd, add=ad))
    assert torch.equal(block(xd.view(1, T, K), zd.view(1, T, E), add=ad.view(1, T, K)).view(T, K), out)

    r = oracle.route(z.astype(np.float64), k, "softmax", True, 1.5)
    n = r["offsets"][-1]
    xf = fake(x, fmt)[r["rows"][:n]]
    h = bf16_round(oracle.grouped(xf, w1, r["offsets"]))
    y = fake(h[:, :F] / (1 + np.exp(-h[:, :F])) * h[:, F:], fmt)
    y = bf16_round(oracle.grouped(y, w2, r["offsets"])) if n else np.zeros((0, K))
    ref = oracle.combine(y, r["positions"], r["weights"], add)
    # h may be the next bf16 value (2^-7) and its code the next E4M3 value (2^-3): of the terms of a
    # product at most, and rarely of many; the 2-norm over a row of them stays within one code's half
    # step (2^-4) of the row's, before the final roundings
    err, size = np.linalg.norm(f64(out) - ref, axis=1), np.linalg.norm(ref - add, axis=1)
    assert (err <= 2.0 ** -4 * size + 2.0 ** -7 * np.linalg.norm(ref, axis=1)).all()
    if T > 4:
        assert torch.equal(out[2], ad[2])


@pytest.mark.parametrize("fmt", ["mxfp8", "fp8_128"])
@pytest.mark.parametrize("T", [3, 150])
def test_expert_mlp_in_a_graph_and_on_streams(fmt, T):
    dev = device()
    rng = np.random.default_rng(T)
    E, k, K, F = 8, 3, 256, 256
    q1, s1, _ = weights(rng, fmt, E, 2 * F, K)
    q2, s2, _ = weights(rng, fmt, E, K, F)
    block = mlp.ExpertMLP(pack(ops, q1, s1, fmt, dev), pack(ops, q2, s2, fmt, dev), k)
    xs = [to_bf16(bf16_round(rng.standard_normal((T, K))), dev) for _ in range(3)]
    zs = [to_dev(rng.standard_normal((T, E)).astype(np.float32), dev) for _ in range(3)]
    want = [block(x, z) for x, z in zip(xs, zs)]
    x, z = xs[0].clone(), zs[0].clone()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = block(x, z)
    for i in (1, 2, 0):
        x.copy_(xs[i])
        z.copy_(zs[i])
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want[i])
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [[], []]
    for _ in range(6):
        for i, st in enumerate(streams):
            with torch.cuda.stream(st):
                got[i].append(block(xs[i], zs[i]))
    torch.cuda.synchronize()
    ops.check()
    for i in range(2):
        assert all(torch.equal(y, want[i]) for y in got[i])


def test_no_tokens():
    dev = device()
    rng = np.random.default_rng(0)
    q1, s1, _ = weights(rng, "mxfp8", 2, 256, 128)
    q2, s2, _ = weights(rng, "mxfp8", 2, 128, 128)
    block = mlp.ExpertMLP(pack(ops, q1, s1, "mxfp8", dev), pack(ops, q2, s2, "mxfp8", dev), 1)
    out = block(torch.empty(0, 128, dtype=torch.bfloat16, device=dev), torch.empty(0, 2, device=dev))
    assert tuple(out.shape) == (0, 128)


def test_tensors_of_another_device(monkeypatch):
    # calls go to the current device's stream: tensors elsewhere are refused
    dev = device()
    rng = np.random.default_rng(0)
    fmt, bf = "fp8_128", torch.bfloat16
    q1, s1, _ = weights(rng, fmt, 2, 256, 128)
    q2, s2, _ = weights(rng, fmt, 2, 128, 128)
    w1, w2 = pack(ops, q1, s1, fmt, dev), pack(ops, q2, s2, fmt, dev)
    x, z = torch.ones(4, 128, dtype=bf, device=dev), torch.zeros(4, 2, device=dev)
    r = ops.route(z, 1)
    y = ops.grouped_linear(x, w2, r.offsets)
    calls = [lambda: ops.quantize_fp8_128(x), lambda: ops.quantize_weights_fp8_128(x), lambda: ops.silu_mul_quantize(x, fmt=fmt),
             lambda: ops.silu_mul_quantize(x, x, fmt=fmt), lambda: ops.linear_fp8_128(x[None].expand(2, 4, 128).contiguous(), w2),
             lambda: ops.grouped_linear(x, w2, r.offsets), lambda: ops.route(z, 1), lambda: ops.combine(y, r),
             lambda: ops.expert_mlp(x, z, w1, w2, 1)]
    for call in calls:
        call()
    for call in (lambda: ops.combine(y, r, add=y.cpu()), lambda: ops.expert_mlp(x, z, w1, w2, 1, add=x.cpu()),
                 lambda: ops.silu_mul_quantize(x, x.cpu(), fmt=fmt), lambda: ops.grouped_linear(x, w2, r.offsets.cpu()),
                 lambda: ops.expert_mlp(x, z.cpu(), w1, w2, 1)):
        with pytest.raises(ValueError, match="CUDA device"):
            call()
    with monkeypatch.context() as m:
        m.setattr(ops, "_current_device", lambda: dev.index + 1 if dev.index is not None else 1)
        for call in calls:
            with pytest.raises(ValueError, match="current"):
                call()
    ops.check()
