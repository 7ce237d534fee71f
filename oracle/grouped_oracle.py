"""Block-128 FP8, products grouped by expert, and expert routing in plain fp64 numpy.

* quantize_b128: one fp32 scale amax / 448 per 128 elements along the last axis,
  codes E4M3(448 x / amax) to nearest even.  For values of at most 8 significant
  bits the fp64 quotient of the exact 448 x is a tie exactly where there is one;
* quantize_weights_b128: one scale per 128 x 128 block;
* grouped: rows [offsets[e], offsets[e + 1]) times w[e]^T;
* route: the k largest logits of each token, ties to the lowest expert, -inf and
  NaN never chosen; rows sorted by (expert, token);
* combine: each token's weighted sum of its rows.
"""

from __future__ import annotations

import math

import numpy as np

from .mx_oracle import e4m3_encode, e4m3_value

BLOCK128 = 128


def _codes_b128(x: np.ndarray, amax: np.ndarray) -> np.ndarray:
    """E4M3 codes of x (fp64) with its block's amax broadcast beside it."""
    safe = np.where((amax > 0) & np.isfinite(amax), amax, 1.0)
    q = e4m3_encode(np.where(np.isfinite(x), x, 0.0) * 448.0 / safe)
    return np.where(np.isfinite(amax), q, 0x7F).astype(np.uint8)


def _scale_b128(amax: np.ndarray) -> np.ndarray:
    with np.errstate(over="ignore", invalid="ignore"):
        s = (amax.astype(np.float32) / np.float32(448.0)).astype(np.float32)
    return np.where(np.isfinite(amax), s, np.float32(np.nan)).astype(np.float32)


def _amax(x: np.ndarray, axis) -> np.ndarray:
    """Largest magnitude; +inf if any element is Inf or NaN."""
    return np.max(np.where(np.isfinite(x), np.abs(x), np.inf), axis=axis)


def quantize_b128(x: np.ndarray) -> tuple[np.ndarray, np.ndarray]:
    """x fp64 [..., K] -> (codes uint8 [..., K], scales fp32 [..., ceil(K / 128)])."""
    K = x.shape[-1]
    kb = -(-K // BLOCK128)
    full = np.zeros((*x.shape[:-1], kb * BLOCK128))
    full[..., :K] = x
    amax = _amax(full.reshape(*x.shape[:-1], kb, BLOCK128), -1)
    return _codes_b128(x, np.repeat(amax, BLOCK128, -1)[..., :K]), _scale_b128(amax)


def quantize_weights_b128(w: np.ndarray) -> tuple[np.ndarray, np.ndarray]:
    """w fp64 [..., N, K] -> (codes, scales fp32 [..., ceil(N / 128), ceil(K / 128)])."""
    N, K = w.shape[-2:]
    nb, kb = -(-N // BLOCK128), -(-K // BLOCK128)
    full = np.zeros((*w.shape[:-2], nb * BLOCK128, kb * BLOCK128))
    full[..., :N, :K] = w
    amax = _amax(full.reshape(*w.shape[:-2], nb, BLOCK128, kb, BLOCK128), (-3, -1))
    wide = np.repeat(np.repeat(amax, BLOCK128, -1)[..., :K], BLOCK128, -2)[..., :N, :]
    return _codes_b128(w, wide), _scale_b128(amax)


def dequantize_b128(q: np.ndarray, s: np.ndarray) -> np.ndarray:
    return e4m3_value(q) * np.repeat(s.astype(np.float64), BLOCK128, -1)[..., :q.shape[-1]]


def dequantize_weights_b128(q: np.ndarray, s: np.ndarray) -> np.ndarray:
    N, K = q.shape[-2:]
    wide = np.repeat(np.repeat(s.astype(np.float64), BLOCK128, -1)[..., :K], BLOCK128, -2)[..., :N, :]
    return e4m3_value(q) * wide


def grouped(x: np.ndarray, w: np.ndarray, offsets, bias: np.ndarray | None = None) -> np.ndarray:
    """fp64 rows [R, K] and weights [E, N, K]; rows of no group are NaN in the result."""
    out = np.full((x.shape[0], w.shape[1]), np.nan)
    for e in range(w.shape[0]):
        lo, hi = int(offsets[e]), int(offsets[e + 1])
        if hi > lo:
            out[lo:hi] = x[lo:hi] @ w[e].T + (0.0 if bias is None else bias[e])
    return out


def route(logits: np.ndarray, k: int, scoring: str = "softmax", renormalize: bool = False, scale: float = 1.0) -> dict:
    """ids, weights (fp64), offsets, rows, positions as the library's route returns them."""
    T, E = logits.shape
    ids = np.full((T, k), -1, dtype=np.int64)
    weights = np.zeros((T, k))
    per_expert: list[list[tuple[int, int]]] = [[] for _ in range(E)]
    for t in range(T):
        z = [float(v) for v in logits[t]]
        able = [e for e in range(E) if not (math.isnan(z[e]) or z[e] == -math.inf)]
        chosen = sorted(able, key=lambda e: (-z[e], e))[:k]
        if not chosen:
            continue
        top = z[chosen[0]]
        total = math.fsum(math.exp(z[e] - top) for e in able)
        w = [math.exp(z[e] - top) / total if scoring == "softmax" else 1.0 / (1.0 + math.exp(min(-z[e], 700.0)))
             for e in chosen]
        s = math.fsum(w)
        if renormalize and s > 0:
            w = [v / s for v in w]
        for j, e in enumerate(chosen):
            ids[t, j], weights[t, j] = e, w[j] * scale
            per_expert[e].append((t, j))
    offsets = np.zeros(E + 1, dtype=np.int64)
    rows = np.full(T * k, -1, dtype=np.int64)
    positions = np.full((T, k), -1, dtype=np.int64)
    at = 0
    for e in range(E):
        for t, j in per_expert[e]:
            rows[at], positions[t, j] = t, at
            at += 1
        offsets[e + 1] = at
    return {"ids": ids, "weights": weights, "offsets": offsets, "rows": rows, "positions": positions}


def combine(y: np.ndarray, positions: np.ndarray, weights: np.ndarray, add: np.ndarray | None = None) -> np.ndarray:
    T, k = positions.shape
    out = np.zeros((T, y.shape[1])) if add is None else add.astype(np.float64).copy()
    for t in range(T):
        for j in range(k):
            if 0 <= positions[t, j] < y.shape[0]:
                out[t] += float(weights[t, j]) * y[positions[t, j]]
    return out
