"""Inputs and tolerances shared by the block-128, grouped and routing tests."""

import numpy as np
import torch

import oracle


def bf16_round(x: np.ndarray) -> np.ndarray:
    """fp64 values of x rounded to bf16."""
    return torch.from_numpy(np.ascontiguousarray(x)).float().to(torch.bfloat16).double().numpy()


def to_bf16(x: np.ndarray, dev) -> torch.Tensor:
    return torch.from_numpy(np.ascontiguousarray(x)).float().to(torch.bfloat16).to(dev)


def to_dev(a: np.ndarray, dev) -> torch.Tensor:
    return torch.from_numpy(np.ascontiguousarray(a)).to(dev)


def f64(t: torch.Tensor) -> np.ndarray:
    return t.detach().double().cpu().numpy()


def weights(rng, fmt: str, *shape):
    """(codes, scales as the library takes them, fp64 values) of random weights."""
    w = bf16_round(rng.standard_normal(shape) * 0.05)
    if fmt == "fp8_128":
        q, s = oracle.quantize_weights_b128(w)
        return q, s, oracle.dequantize_weights_b128(q, s)
    q, s = oracle.quantize(w)
    return q, s, oracle.dequantize(q, s)


def fake(x: np.ndarray, fmt: str) -> np.ndarray:
    """x quantised and back, fp64."""
    if fmt == "fp8_128":
        return oracle.dequantize_b128(*oracle.quantize_b128(x))
    return oracle.dequantize(*oracle.quantize(x))


def codes(x: np.ndarray, fmt: str):
    return oracle.quantize_b128(x) if fmt == "fp8_128" else oracle.quantize(x)


def pack(ops, q: np.ndarray, s: np.ndarray, fmt: str, dev):
    q_d, s_d = to_dev(q, dev), to_dev(s, dev)
    return ops.process_weights_fp8_128(q_d, s_d) if fmt == "fp8_128" else ops.process_weights(q_d, s_d)


def product_bound(x: np.ndarray, w: np.ndarray, ref: np.ndarray) -> np.ndarray:
    """How far a bf16 product of fp64-valued x [R, K] and w [N, K] may be from ref.

    One rounding to bf16: 2^-8 |out|.  fp32 sums of K products in any order, each
    addition off by at most 2^-23 (tensor cores may truncate) of a partial sum that
    is at most S = sum |x w|, then for each of the K / 128 blocks a scale product
    and a multiply-add (2^-24 each), and the bias: (K + K / 64 + 2) 2^-23 S, with
    (1 + 2^-8) for the rounding of a value that is itself off.
    """
    K = x.shape[-1]
    S = np.abs(x) @ np.abs(w).swapaxes(-1, -2)
    off = (K + K / 64 + 2) * 2.0 ** -23 * (S + np.abs(ref))
    return 2.0 ** -8 * np.abs(ref) + (1 + 2.0 ** -8) * off


def assert_product(out: torch.Tensor, ref: np.ndarray, bound: np.ndarray, what: str = "") -> None:
    got = f64(out)
    assert got.shape == ref.shape
    bad = ~(np.abs(got - ref) <= bound)
    if bad.any():
        i = tuple(np.argwhere(bad)[0])
        raise AssertionError(f"{what}: {int(bad.sum())}/{bad.size} off, first at {i}: {got[i]} for {ref[i]} +- {bound[i]}")


def offsets_of(counts) -> np.ndarray:
    return np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
