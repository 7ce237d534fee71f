"""CPU oracle of the 4-bit formats, the RMS norm and the gated activation:
test infrastructure only, plain numpy, no code shared with the library.

MXFP4 (OCP MX v1.0, sections 5.3.3 and 6.3): E2M1 elements, one E8M0 scale
2**(floor(log2 amax) - 2) per 32.  NVFP4: E2M1 elements, one E4M3 scale per 16,
one fp32 scale g per tensor; its rule is stated in fp32 steps and follows them
for every g >= 0 (g = 0, the amax of an all-zero tensor: the value is 0).
"""

from __future__ import annotations

import numpy as np

from .mx_oracle import e4m3_encode, e4m3_value, e8m0_value, quantize

E2M1_VALUES = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
BLOCKS = {"mxfp8": 32, "mxfp4": 32, "nvfp4": 16}


def e2m1_encode(x: np.ndarray) -> np.ndarray:
    """Codes (0..15) of the nearest E2M1 value, ties to the even code, saturating."""
    x = np.asarray(x, dtype=np.float64)
    a = np.minimum(np.abs(x), 6.0)
    mids = (E2M1_VALUES[1:] + E2M1_VALUES[:-1]) / 2
    lo = np.searchsorted(mids, a, side="left")   # ties stay below
    hi = np.searchsorted(mids, a, side="right")  # ties go above
    code = np.where(lo % 2 == 0, lo, hi)
    return (code | np.where(np.signbit(x), 8, 0)).astype(np.uint8)


def e2m1_value(code: np.ndarray) -> np.ndarray:
    code = np.asarray(code)
    v = E2M1_VALUES[code & 7]
    return np.where(code & 8, -v, v)


def pack(codes: np.ndarray) -> np.ndarray:
    """Codes [..., K] -> bytes [..., K/2], the even element in the low half."""
    return (codes[..., 0::2] | (codes[..., 1::2] << 4)).astype(np.uint8)


def unpack(q: np.ndarray) -> np.ndarray:
    return np.stack([q & 15, q >> 4], axis=-1).reshape(*q.shape[:-1], -1)


def quantize4(x: np.ndarray, fmt: str, g: float = 1.0):
    """x [..., K] -> (codes [..., K] one per byte, scale bytes [..., K/block])."""
    x = np.asarray(x, dtype=np.float64)
    n = BLOCKS[fmt]
    xb = x.reshape(*x.shape[:-1], x.shape[-1] // n, n)
    bad = ~np.isfinite(xb).all(-1)
    safe = np.where(bad[..., None], 0.0, xb)
    amax = np.abs(safe).max(-1)
    if fmt == "mxfp4":
        with np.errstate(divide="ignore"):
            e = np.where(amax > 0, np.floor(np.log2(np.where(amax > 0, amax, 1.0))), -1000.0) - 2
        # floor(log2) from the bits: log2 rounds near powers of two
        e = np.where(amax > 0, np.frexp(np.where(amax > 0, amax, 1.0))[1] - 1 - 2, e)
        e = np.clip(e, -127, 127)
        s = np.where(bad, 0xFF, e + 127).astype(np.uint8)
        t = safe / np.exp2(e)[..., None]
    else:
        f = np.float32
        with np.errstate(divide="ignore", over="ignore", invalid="ignore"):
            six_g = np.maximum(f(6.0) * f(g), f(2.0 ** -149))  # a zero block is 0 even for g = 0
            s = e4m3_encode((amax.astype(f) / six_g).astype(np.float64)).astype(np.uint8)
        unit = e4m3_value(s).astype(f) * f(g)
        with np.errstate(divide="ignore", over="ignore"):
            inv = f(1.0) / unit
        inv = np.where((unit > 0) & np.isfinite(inv), inv, f(0.0)).astype(f)
        with np.errstate(over="ignore"):
            t = (safe.astype(f) * inv[..., None]).astype(np.float64)
        s = np.where(bad, 0x7F, s).astype(np.uint8)
    codes = np.where(bad[..., None], 0, e2m1_encode(t)).astype(np.uint8)
    return codes.reshape(x.shape), s


def dequantize4(codes: np.ndarray, s: np.ndarray, fmt: str, g: float = 1.0) -> np.ndarray:
    n = BLOCKS[fmt]
    v = e2m1_value(codes).reshape(*codes.shape[:-1], codes.shape[-1] // n, n)
    unit = e8m0_value(s) if fmt == "mxfp4" else e4m3_value(s) * float(np.float32(g))
    return (v * unit[..., None]).reshape(codes.shape)


def quantize_any(x: np.ndarray, fmt: str, g: float = 1.0):
    """(codes one per byte, scale bytes) in MXFP8, MXFP4 or NVFP4."""
    return quantize(x) if fmt == "mxfp8" else quantize4(x, fmt, g)


def rmsnorm(x, weight, residual=None, eps=1e-6):
    """(t, y) in fp64."""
    t = np.asarray(x, dtype=np.float64)
    if residual is not None:
        t = t + np.asarray(residual, dtype=np.float64)
    return t, t / np.sqrt(np.mean(t * t, axis=-1, keepdims=True) + eps) * np.asarray(weight, dtype=np.float64)


def silu_mul(gate, up):
    gate = np.asarray(gate, dtype=np.float64)
    with np.errstate(over="ignore"):
        return gate / (1.0 + np.exp(-gate)) * np.asarray(up, dtype=np.float64)
