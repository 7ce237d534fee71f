"""Thin ctypes binding over libmxfp8.so (include/mxfp8.h).

Argument marshalling only: every step of the layer runs in the library's CUDA
kernels.  PyTorch provides device memory and the current stream.  There is no
fallback: if the library is missing or the GPU is not sm_103, calls raise.

Shapes follow the vLLM pages: "CompressedTensorsW8A8Mxfp8.create_weights"
(weight [N, K] E4M3, weight_scale [N, K // 32] uint8) and
"AiterFlyDSLMxfp8LinearKernel.apply_weights" (x [..., K] bf16 or a
pre-quantised x_q [..., K] with row-major scales [..., K // 32]; output
[..., N] in bf16, plus bias).
"""

from __future__ import annotations

import ctypes
import dataclasses
import functools
import os

import numpy as np
import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libmxfp8.so")
BLOCK = 32

_STATUS = {0: "MXFP8_OK", 1: "MXFP8_ERR_INVALID_ARG", 2: "MXFP8_ERR_UNSUPPORTED",
           3: "MXFP8_ERR_ARCH", 4: "MXFP8_ERR_CUDA", 5: "MXFP8_ERR_TIMEOUT"}

# name -> (restype, argtypes), mirroring include/mxfp8.h
_P, _I64, _U64, _INT = ctypes.c_void_p, ctypes.c_int64, ctypes.c_uint64, ctypes.c_int
_SIZE_P = ctypes.POINTER(ctypes.c_size_t)
SIGNATURES = {
    "mxfp8_last_error": (ctypes.c_char_p, []),
    "mxfp8_version": (_INT, []),
    "mxfp8_quantize": (_INT, [_P, _I64, _I64, _P, _P, _P]),
    "mxfp8_packed_sizes": (_INT, [_I64, _I64, _I64, _SIZE_P, _SIZE_P]),
    "mxfp8_process_weights": (_INT, [_P, _P, _I64, _I64, _I64, _P, _P, _P]),
    "mxfp8_unpack_scales": (_INT, [_P, _I64, _I64, _I64, _P, _P]),
    "mxfp8_workspace_size": (_INT, [_I64, _I64, _I64, _I64, _INT, _SIZE_P]),
    "mxfp8_linear": (_INT, [_P, _P, _P, _I64, _I64, _I64, _I64, _P, _P, _P, _P, _P,
                            ctypes.c_size_t, _P]),
    "mxfp8_linear_path": (_INT, [_INT, _P, _P, _P, _I64, _I64, _I64, _I64, _P, _P, _P, _P,
                                 _P, ctypes.c_size_t, _P]),
    "mxfp8_quantize_packed": (_INT, [_P, _I64, _I64, _I64, _P, _P, _P]),
    "mxfp8_pack_scales": (_INT, [_P, _I64, _I64, _I64, _P, _P]),
    "mxfp8_gemm_packed": (_INT, [_P, _P, _I64, _I64, _I64, _I64, _P, _P, _P, _P, _P]),
    "mxfp8_linear_noalloc": (_INT, [_P, _I64, _I64, _I64, _I64, _P, _P, _P, _P, _P]),
    "mxfp8_linear_quantized_out": (_INT, [_P, _P, _P, _I64, _I64, _I64, _I64, _P, _P, _P, _P, _P, _P,
                                          _P, ctypes.c_size_t, _P]),
    "mxfp8_gemm_packed_quantized_out": (_INT, [_P, _P, _I64, _I64, _I64, _I64, _P, _P, _P, _P, _P, _P,
                                               _P]),
    "mxfp8_blob_size": (_INT, [_I64, _I64, _I64, _INT, _SIZE_P]),
    "mxfp8_weights_serialize": (_INT, [_P, _P, _I64, _I64, _I64, _INT, _INT, _P, ctypes.c_size_t]),
    "mxfp8_weights_deserialize": (_INT, [_P, ctypes.c_size_t, ctypes.POINTER(ctypes.c_int64),
                                         ctypes.POINTER(ctypes.c_int64), ctypes.POINTER(ctypes.c_int64),
                                         ctypes.POINTER(ctypes.c_int), ctypes.POINTER(ctypes.c_int),
                                         _SIZE_P, _SIZE_P]),
    "mxfp8_quantize_weights": (_INT, [_P, _I64, _I64, _INT, _P, _P, _P]),
    "mxfp8_packed_sizes_fmt": (_INT, [_INT, _I64, _I64, _I64, _SIZE_P, _SIZE_P]),
    "mxfp8_process_weights_fmt": (_INT, [_INT, _P, _P, _I64, _I64, _I64, _P, _P, _P]),
    "mxfp8_linear_fmt": (_INT, [_INT, _INT, _P, _P, _P, _I64, _I64, _I64, _I64, _P, _P, _P, _P, _P,
                                ctypes.c_size_t, _P]),
    "mxfp8_fp4_quantize": (_INT, [_INT, _P, _I64, _I64, _P, _P, _P, _P]),
    "mxfp8_fp4_quantize_packed": (_INT, [_INT, _P, _I64, _I64, _I64, _P, _P, _P, _P]),
    "mxfp8_fp4_unpack": (_INT, [_P, _I64, _P, _P]),
    "mxfp8_fp4_packed_sizes": (_INT, [_INT, _I64, _I64, _I64, _SIZE_P, _SIZE_P]),
    "mxfp8_fp4_process_weights": (_INT, [_INT, _P, _P, _I64, _I64, _I64, _P, _P, _P]),
    "mxfp8_fp4_workspace_size": (_INT, [_INT, _I64, _I64, _I64, _I64, _INT, _SIZE_P]),
    "mxfp8_fp4_product_workspace_size": (_INT, [_INT, _I64, _I64, _I64, _I64, _SIZE_P]),
    "mxfp8_fp4_linear": (_INT, [_INT, _P, _P, _P, _P, _I64, _I64, _I64, _I64, _P, _P, _P, _P, _P, _P,
                                ctypes.c_size_t, _P]),
    "mxfp8_fp4_gemm_packed": (_INT, [_INT, _P, _P, _P, _I64, _I64, _I64, _I64, _P, _P, _P, _P, _P, _P,
                                     ctypes.c_size_t, _P]),
    "mxfp8_rmsnorm_quantize": (_INT, [_INT, _P, _I64, _P, _I64, _INT, _P, _P, ctypes.c_float, _P, _I64, _I64,
                                      _P, _P, _INT, _P, _P]),
    "mxfp8_silu_mul_quantize": (_INT, [_INT, _P, _I64, _P, _I64, _P, _I64, _I64, _P, _P, _INT, _P]),
    "mxfp8_gated_mlp_workspace_size": (_INT, [_INT, _I64, _I64, _I64, _SIZE_P]),
    "mxfp8_gated_mlp": (_INT, [_INT, _P, _I64, _P, _I64, _INT, _P, _P, ctypes.c_float, _I64, _I64, _I64, _P, _P, _P,
                               _P, _P, _P, _P, _P, _P, _P, ctypes.c_size_t, _P]),
    "mxfp8_check": (_INT, [_P]),
    "mxfp8_debug_expire_wait": (_INT, [_U64, _P]),
}

_lib = None

# weight element formats (MXFP8_WFMT_*): E4M3 (MXFP8) and the MXFP6 E2M3 / E3M2
WFMT = {"e4m3": 0, "e2m3": 1, "e3m2": 2}

# formats of the quantising calls (MXFP8_QFMT_*) and their block lengths; the
# 4-bit ones are also weight formats of linear_fp4
QFMT = {"mxfp8": 0, "mxfp4": 1, "nvfp4": 2}
QBLOCK = {"mxfp8": 32, "mxfp4": 32, "nvfp4": 16}


class MxStatusError(RuntimeError):
    def __init__(self, status: int, text: str):
        self.status = status
        super().__init__(f"{_STATUS.get(status, status)}: {text}")


def load(path: str = LIB_PATH) -> ctypes.CDLL:
    """Load libmxfp8.so (once).  Raises if it has not been built."""
    global _lib
    if _lib is None:
        if not os.path.exists(path):
            raise RuntimeError(f"{path} is missing: build it with "
                               "`python -m mxfp8_block_scaled_02_gb300.build`")
        lib = ctypes.CDLL(path)
        for name, (res, args) in SIGNATURES.items():
            fn = getattr(lib, name)
            fn.restype = res
            fn.argtypes = args
        _lib = lib
    return _lib


def _check(status: int) -> None:
    if status != 0:
        raise MxStatusError(status, load().mxfp8_last_error().decode())


def _stream() -> int:
    # the handle alone: torch.cuda.current_stream() builds a Stream object
    # (2.9 us per call on the Grace host, of ~10 for a whole call)
    if torch.cuda.is_initialized():
        return torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice())
    return torch.cuda.current_stream().cuda_stream


def _ptr(t: torch.Tensor | None) -> int | None:
    return None if t is None else t.data_ptr()


def _bytes(t: torch.Tensor) -> torch.Tensor:
    """Same memory viewed as uint8 (E4M3 / E8M0 tensors are passed as bytes)."""
    return t if t.dtype == torch.uint8 else t.view(torch.uint8)


def _require_cuda(*ts: torch.Tensor | None) -> None:
    for t in ts:
        if t is not None:
            if not t.is_cuda:
                raise ValueError("tensors must be on a CUDA device")
            if not t.is_contiguous():
                raise ValueError("tensors must be contiguous")


def _aligned16(t: torch.Tensor | None) -> torch.Tensor | None:
    """The same values at a 16-byte aligned address (every pointer the ABI takes
    must be; a view into a larger tensor may not be), copied only if needed."""
    if t is None or t.data_ptr() % 16 == 0:
        return t
    return t.clone(memory_format=torch.contiguous_format)


def quantize(x: torch.Tensor) -> tuple[torch.Tensor, torch.Tensor]:
    """bf16 x [..., K] -> (x_q uint8 E4M3 [..., K], x_scale uint8 E8M0 [..., K/32])."""
    if x.dtype != torch.bfloat16:
        raise TypeError("x must be bfloat16")
    _require_cuda(x)
    x = _aligned16(x)
    K = x.shape[-1]
    rows = x.numel() // K if K else 0
    q = torch.empty(x.shape, dtype=torch.uint8, device=x.device)
    s = torch.empty((*x.shape[:-1], K // BLOCK), dtype=torch.uint8, device=x.device)
    _check(load().mxfp8_quantize(_ptr(x), rows, K, _ptr(q), _ptr(s), _stream()))
    return q, s


def packed_sizes(B: int, N: int, K: int, fmt: str = "e4m3") -> tuple[int, int]:
    wb, sb = ctypes.c_size_t(), ctypes.c_size_t()
    _check(load().mxfp8_packed_sizes_fmt(WFMT[fmt], B, N, K, ctypes.byref(wb), ctypes.byref(sb)))
    return wb.value, sb.value


def quantize_weights(w: torch.Tensor, fmt: str = "e4m3") -> tuple[torch.Tensor, torch.Tensor]:
    """bf16 weights [..., K] -> (codes uint8 [..., K], one per byte; scales uint8
    [..., K/32]) in ``fmt`` ("e4m3", or the MXFP6 "e2m3" / "e3m2")."""
    if w.dtype != torch.bfloat16:
        raise TypeError("w must be bfloat16")
    _require_cuda(w)
    w = _aligned16(w)
    K = w.shape[-1]
    rows = w.numel() // K if K else 0
    q = torch.empty(w.shape, dtype=torch.uint8, device=w.device)
    s = torch.empty((*w.shape[:-1], K // BLOCK), dtype=torch.uint8, device=w.device)
    _check(load().mxfp8_quantize_weights(_ptr(w), rows, K, WFMT[fmt], _ptr(q), _ptr(s), _stream()))
    return q, s


@dataclasses.dataclass
class PackedWeights:
    """Weights after the one-time repack (process_weights, process_weights_fp4):
    element bytes and scale atoms.  A product may read these two before the
    kernel ahead of it in the stream has finished, so they are not to be another
    call's outputs (codes that a norm or activation wrote); every other input may."""

    w_packed: torch.Tensor   # uint8, B*N*K bytes (3BNK/4 for packed FP6, BNK/2 for FP4)
    sf_packed: torch.Tensor  # uint8, packed scale atoms
    B: int
    N: int
    K: int
    batched: bool
    fmt: str = "e4m3"        # weight element format: "e4m3", "e2m3", "e3m2", or "mxfp4" / "nvfp4"
    tensor_scale: torch.Tensor | None = None  # NVFP4: fp32, one element


def process_weights(w_q: torch.Tensor, w_scale: torch.Tensor, fmt: str = "e4m3") -> PackedWeights:
    """w_q [N, K] or [B, N, K] (uint8 or float8_e4m3fn; for ``fmt`` "e2m3" /
    "e3m2" one FP6 code per byte), w_scale [..., K/32] uint8.

    A checkpoint may store its scales padded (more rows than N or more blocks
    than K/32, as the aiter_flydsl page's process_weights_after_loading slices
    them with ``[:N, :K // 32]``): the padding is sliced off here and the
    scales copied to a dense, aligned tensor before the repack.
    """
    if w_q.dim() not in (2, 3):
        raise ValueError("w_q must be [N, K] or [B, N, K]")
    batched = w_q.dim() == 3
    B = w_q.shape[0] if batched else 1
    N, K = w_q.shape[-2], w_q.shape[-1]
    if K % BLOCK:
        raise ValueError(f"K={K} is not a multiple of {BLOCK}")
    if (w_scale.dim() != w_q.dim() or tuple(w_scale.shape[:-2]) != tuple(w_q.shape[:-2])
            or w_scale.shape[-2] < N or w_scale.shape[-1] < K // BLOCK):
        raise ValueError(f"weight scale {tuple(w_scale.shape)} does not match weight {tuple(w_q.shape)}")
    w_scale = w_scale[..., :N, :K // BLOCK]
    if not w_scale.is_contiguous():
        w_scale = w_scale.contiguous()
    w_q, w_scale = _aligned16(w_q), _aligned16(w_scale)
    _require_cuda(w_q, w_scale)
    wb, sb = packed_sizes(B, N, K, fmt)
    wp = torch.empty(wb, dtype=torch.uint8, device=w_q.device)
    sp = torch.empty(sb, dtype=torch.uint8, device=w_q.device)
    _check(load().mxfp8_process_weights_fmt(WFMT[fmt], _ptr(_bytes(w_q)), _ptr(_bytes(w_scale)), B, N, K,
                                            _ptr(wp), _ptr(sp), _stream()))
    return PackedWeights(wp, sp, B, N, K, batched, fmt)


def _not_fp4(pw: PackedWeights, what: str) -> None:
    if pw.fmt not in WFMT:
        raise ValueError(f"{what} does not take {pw.fmt} weights; use linear_fp4 / gemm_packed_fp4")


def save_packed(pw: PackedWeights) -> bytes:
    """The packed weights as one self-describing blob (mxfp8_weights_serialize):
    a versioned, checksummed header, then the w_packed and sf_packed bytes.
    Write it to a file once; load_packed restores it without repacking."""
    _not_fp4(pw, "save_packed")
    w = np.ascontiguousarray(pw.w_packed.detach().cpu().numpy())
    sf = np.ascontiguousarray(pw.sf_packed.detach().cpu().numpy())
    n = ctypes.c_size_t()
    _check(load().mxfp8_blob_size(pw.B, pw.N, pw.K, WFMT[pw.fmt], ctypes.byref(n)))
    if (w.size, sf.size) != packed_sizes(pw.B, pw.N, pw.K, pw.fmt):
        raise ValueError("packed tensors do not have the sizes of (B, N, K)")
    blob = np.empty(n.value, dtype=np.uint8)
    _check(load().mxfp8_weights_serialize(w.ctypes.data, sf.ctypes.data, pw.B, pw.N, pw.K, WFMT[pw.fmt],
                                          int(pw.batched), blob.ctypes.data, blob.size))
    return blob.tobytes()


def load_packed(blob: bytes | bytearray | memoryview, device: torch.device | str) -> PackedWeights:
    """PackedWeights from a blob written by save_packed (checked by
    mxfp8_weights_deserialize: format, layout, sizes and both checksums),
    copied to ``device``."""
    buf = np.frombuffer(blob, dtype=np.uint8)
    B, N, K = ctypes.c_int64(), ctypes.c_int64(), ctypes.c_int64()
    fmt, batched = ctypes.c_int(), ctypes.c_int()
    wo, so = ctypes.c_size_t(), ctypes.c_size_t()
    _check(load().mxfp8_weights_deserialize(buf.ctypes.data, buf.size, ctypes.byref(B), ctypes.byref(N),
                                            ctypes.byref(K), ctypes.byref(fmt), ctypes.byref(batched),
                                            ctypes.byref(wo), ctypes.byref(so)))
    name = {v: k for k, v in WFMT.items()}[fmt.value]
    wb, sb = packed_sizes(B.value, N.value, K.value, name)
    w = torch.from_numpy(buf[wo.value:wo.value + wb].copy()).to(device)
    sf = torch.from_numpy(buf[so.value:so.value + sb].copy()).to(device)
    return PackedWeights(w, sf, B.value, N.value, K.value, bool(batched.value), name)


def unpack_scales(pw: PackedWeights) -> torch.Tensor:
    _not_fp4(pw, "unpack_scales")
    out = torch.empty((pw.B, pw.N, pw.K // BLOCK), dtype=torch.uint8, device=pw.sf_packed.device)
    _check(load().mxfp8_unpack_scales(_ptr(pw.sf_packed), pw.B, pw.N, pw.K, _ptr(out), _stream()))
    return out if pw.batched else out[0]


def workspace_size(B: int, M: int, N: int, K: int, quantized: bool) -> int:
    n = ctypes.c_size_t()
    _check(load().mxfp8_workspace_size(B, M, N, K, int(quantized), ctypes.byref(n)))
    return n.value


def _linear_rows(x: torch.Tensor, pw: PackedWeights, bias: torch.Tensor | None,
                 x_scale: torch.Tensor | None, out: torch.Tensor | None) -> int:
    """Check x (and x_scale, bias, out) against the packed weights; returns M,
    the rows per batch.  Shared by every linear entry point, so that none of
    them hands the library a buffer shorter than the sizes it is told."""
    _not_fp4(pw, "this call")
    quantized = x_scale is not None
    if not quantized and x.dtype != torch.bfloat16:
        raise TypeError("x must be bfloat16 (or pass x_scale with a pre-quantised x)")
    if quantized and x.dtype not in (torch.uint8, torch.float8_e4m3fn):
        raise TypeError("a pre-quantised x must be uint8 or float8_e4m3fn E4M3 codes")
    _require_cuda(x, x_scale, bias, out)
    if x.dim() < 1:
        raise ValueError("x must have a K dimension")
    K = x.shape[-1]
    if K != pw.K:
        raise ValueError(f"x has K={K}, weights have K={pw.K}")
    if pw.batched:
        if x.dim() != 3 or x.shape[0] != pw.B:
            raise ValueError("batched weights need x of shape [B, M, K]")
        M = x.shape[1]
    else:
        M = x.numel() // K if K else 0
    if quantized and (x_scale.dtype not in (torch.uint8, torch.float8_e8m0fnu)
                      or tuple(x_scale.shape) != (*x.shape[:-1], K // BLOCK)):
        raise ValueError(f"MXFP8 activation scale {tuple(x_scale.shape)} for {tuple(x.shape)}")
    if bias is not None and (bias.dtype != torch.bfloat16 or tuple(bias.shape) != (pw.N,)):
        raise ValueError("bias must be bf16 [N]")
    if out is not None and (out.dtype != torch.bfloat16 or out.numel() != pw.B * M * pw.N):
        raise ValueError(f"out must be bf16 with {pw.B * M * pw.N} elements")
    return M


def linear(x: torch.Tensor, pw: PackedWeights, bias: torch.Tensor | None = None,
           x_scale: torch.Tensor | None = None, *, path: int = 0,
           out: torch.Tensor | None = None, workspace: torch.Tensor | None = None) -> torch.Tensor:
    """MXFP8 linear layer.

    ``x`` is bf16 ``[..., K]`` (quantised inside the call), or with ``x_scale``
    given, the pre-quantised E4M3 ``x_q [..., K]`` with row-major scales
    ``[..., K/32]``.  For batched weights (``[B, N, K]``) x is ``[B, M, K]``.
    Returns bf16 ``[..., N]``.  ``path`` forces the small-M (1) or large-M (2)
    kernel path, the large-M path on CTA-pair tiles (3), the large-M kernels
    without the small-M one (4), or the GEMM that quantises bf16 x itself (5);
    0 lets the library choose.
    """
    quantized = x_scale is not None
    M = _linear_rows(x, pw, bias, x_scale, out)
    K = pw.K
    x, x_scale, bias = _aligned16(x), _aligned16(x_scale), _aligned16(bias)
    if out is None:
        out = torch.empty((*x.shape[:-1], pw.N), dtype=torch.bfloat16, device=x.device)
    if M == 0:
        return out
    ws_bytes = workspace_size(pw.B, M, pw.N, K, quantized)
    if workspace is None:
        workspace = torch.empty(max(ws_bytes, 1), dtype=torch.uint8, device=x.device)
    xb = None if quantized else x
    xq = _bytes(x) if quantized else None
    _check(load().mxfp8_linear_fmt(path, WFMT[pw.fmt], _ptr(xb), _ptr(xq), _ptr(x_scale), pw.B, M, pw.N, K,
                                   _ptr(pw.w_packed), _ptr(pw.sf_packed), _ptr(bias), _ptr(out),
                                   _ptr(workspace), workspace.numel(), _stream()))
    return out


def _mxfp8_only(pa: PackedActivation, what: str) -> None:
    if pa.fmt != "mxfp8":
        raise ValueError(f"{what} takes MXFP8 activations only (these are {pa.fmt}); use gemm_packed_fp4")


def _e4m3_only(pw: PackedWeights, what: str) -> None:
    if pw.fmt != "e4m3":
        raise ValueError(f"{what} takes E4M3 weights only (these are {pw.fmt}); use "
                         f"{'linear' if pw.fmt in WFMT else 'linear_fp4'}")


@dataclasses.dataclass
class PackedActivation:
    """Activations quantised straight into the GEMM's operand layout."""

    x_q: torch.Tensor        # uint8 [B, M, K] ([B, M, K/2] in the 4-bit formats)
    sf_packed: torch.Tensor  # uint8 packed scale atoms
    B: int
    M: int
    K: int
    fmt: str = "mxfp8"       # "mxfp8", or "mxfp4" / "nvfp4" (gemm_packed_fp4)
    tensor_scale: torch.Tensor | None = None  # NVFP4: fp32, one element


def quantize_packed(x: torch.Tensor, B: int = 1, *, x_q: torch.Tensor | None = None,
                    sf_packed: torch.Tensor | None = None) -> PackedActivation:
    """bf16 x ([M, K], or [B, M, K] with B given) -> E4M3 codes + packed scales."""
    if x.dtype != torch.bfloat16:
        raise TypeError("x must be bfloat16")
    _require_cuda(x)
    x = _aligned16(x)
    K = x.shape[-1]
    M = x.numel() // (K * B)
    if x_q is None:
        x_q = torch.empty((B, M, K), dtype=torch.uint8, device=x.device)
    if sf_packed is None:
        sf_packed = torch.empty(packed_sizes(B, max(M, 1), K)[1], dtype=torch.uint8, device=x.device)
    _check(load().mxfp8_quantize_packed(_ptr(x), B, M, K, _ptr(x_q), _ptr(sf_packed), _stream()))
    return PackedActivation(x_q, sf_packed, B, M, K)


def pack_scales(scale: torch.Tensor, B: int = 1) -> torch.Tensor:
    """Row-major E8M0 scales [B, R, K/32] (or [R, K/32]) -> packed atoms."""
    _require_cuda(scale)
    scale = _aligned16(scale)
    KB = scale.shape[-1]
    R = scale.numel() // (KB * B)
    out = torch.empty(packed_sizes(B, R, KB * BLOCK)[1], dtype=torch.uint8, device=scale.device)
    _check(load().mxfp8_pack_scales(_ptr(_bytes(scale)), B, R, KB * BLOCK, _ptr(out), _stream()))
    return out


def gemm_packed(pa: PackedActivation, pw: PackedWeights, bias: torch.Tensor | None = None,
                out: torch.Tensor | None = None) -> torch.Tensor:
    """The block-scaled GEMM + bias epilogue alone; returns bf16 [B, M, N]."""
    _e4m3_only(pw, "gemm_packed")
    _mxfp8_only(pa, "gemm_packed")
    if pa.K != pw.K or pa.B != pw.B:
        raise ValueError("activation and weights disagree on K or B")
    _require_cuda(bias, out)
    if out is not None and (out.dtype != torch.bfloat16 or out.numel() != pa.B * pa.M * pw.N):
        raise ValueError(f"out must be bf16 with {pa.B * pa.M * pw.N} elements")
    if out is None:
        out = torch.empty((pa.B, pa.M, pw.N), dtype=torch.bfloat16, device=pa.x_q.device)
    _check(load().mxfp8_gemm_packed(_ptr(pa.x_q), _ptr(pa.sf_packed), pa.B, pa.M, pw.N, pa.K,
                                    _ptr(pw.w_packed), _ptr(pw.sf_packed), _ptr(bias), _ptr(out),
                                    _stream()))
    return out


def _hand_off_buffers(B: int, M: int, N: int, device) -> PackedActivation:
    y_q = torch.empty((B, M, N), dtype=torch.uint8, device=device)
    y_sf = torch.empty(packed_sizes(B, max(M, 1), N)[1], dtype=torch.uint8, device=device)
    return PackedActivation(y_q, y_sf, B, M, N)


def linear_quantized_out(x: torch.Tensor, pw: PackedWeights, bias: torch.Tensor | None = None,
                         x_scale: torch.Tensor | None = None, *, bf16_out: bool = True,
                         workspace: torch.Tensor | None = None
                         ) -> tuple[torch.Tensor | None, PackedActivation]:
    """MXFP8 linear layer that also hands its output on quantised
    (mxfp8_linear_quantized_out): returns (bf16 out or None, y as a
    PackedActivation that gemm_packed / gemm_packed_quantized_out take as x)."""
    _e4m3_only(pw, "linear_quantized_out")
    M = _linear_rows(x, pw, bias, x_scale, None)
    quantized = x_scale is not None
    x, x_scale, bias = _aligned16(x), _aligned16(x_scale), _aligned16(bias)
    out = torch.empty((*x.shape[:-1], pw.N), dtype=torch.bfloat16, device=x.device) if bf16_out else None
    y = _hand_off_buffers(pw.B, M, pw.N, x.device)
    if M == 0:
        return out, y
    if workspace is None:
        workspace = torch.empty(max(workspace_size(pw.B, M, pw.N, pw.K, quantized), 1), dtype=torch.uint8,
                                device=x.device)
    xb = None if quantized else x
    xq = _bytes(x) if quantized else None
    _check(load().mxfp8_linear_quantized_out(_ptr(xb), _ptr(xq), _ptr(x_scale), pw.B, M, pw.N, pw.K,
                                             _ptr(pw.w_packed), _ptr(pw.sf_packed), _ptr(bias), _ptr(out),
                                             _ptr(y.x_q), _ptr(y.sf_packed), _ptr(workspace),
                                             workspace.numel(), _stream()))
    return out, y


def gemm_packed_quantized_out(pa: PackedActivation, pw: PackedWeights, bias: torch.Tensor | None = None,
                              *, bf16_out: bool = True) -> tuple[torch.Tensor | None, PackedActivation]:
    """gemm_packed whose output is also handed on quantised
    (mxfp8_gemm_packed_quantized_out): the middle layer of a chain."""
    _e4m3_only(pw, "gemm_packed_quantized_out")
    _mxfp8_only(pa, "gemm_packed_quantized_out")
    if pa.K != pw.K or pa.B != pw.B:
        raise ValueError("activation and weights disagree on K or B")
    _require_cuda(bias)
    out = torch.empty((pa.B, pa.M, pw.N), dtype=torch.bfloat16, device=pa.x_q.device) if bf16_out else None
    y = _hand_off_buffers(pa.B, pa.M, pw.N, pa.x_q.device)
    _check(load().mxfp8_gemm_packed_quantized_out(_ptr(pa.x_q), _ptr(pa.sf_packed), pa.B, pa.M, pw.N, pa.K,
                                                  _ptr(pw.w_packed), _ptr(pw.sf_packed), _ptr(bias), _ptr(out),
                                                  _ptr(y.x_q), _ptr(y.sf_packed), _stream()))
    return out, y


NOALLOC_SCRATCH_BYTES = 32 << 20


def linear_noalloc(x: torch.Tensor, pw: PackedWeights, bias: torch.Tensor | None = None,
                   out: torch.Tensor | None = None) -> torch.Tensor:
    """bf16 linear that allocates no device workspace (mxfp8_linear_noalloc).

    For callers that cannot allocate device memory: the library's fixed
    32 MiB scratch array holds the quantised activations, so B*M*K is limited
    (the call raises MXFP8_ERR_UNSUPPORTED beyond it).  Calls that overlap on
    the GPU share that array and race.  Only ``out`` is allocated here when it
    is not given.
    """
    _e4m3_only(pw, "linear_noalloc")
    M = _linear_rows(x, pw, bias, None, out)
    K = pw.K
    x, bias = _aligned16(x), _aligned16(bias)
    if out is None:
        out = torch.empty((*x.shape[:-1], pw.N), dtype=torch.bfloat16, device=x.device)
    if M == 0:
        return out
    _check(load().mxfp8_linear_noalloc(_ptr(x), pw.B, M, pw.N, K, _ptr(pw.w_packed),
                                       _ptr(pw.sf_packed), _ptr(bias), _ptr(out), _stream()))
    return out


# ------------------------------------------------------------------ 4-bit layer (MXFP4, NVFP4)
# On the Grace host a short call costs as much in Python as in its launches, so
# the functions below look things up once and call few helpers.
_BF16, _F32, _U8, _E4M3 = torch.bfloat16, torch.float32, torch.uint8, torch.float8_e4m3fn
# (MXFP8_QFMT code, elements per code byte, block length) of the quantising formats
_QSPEC = {"mxfp8": (0, 1, 32), "mxfp4": (1, 2, 32), "nvfp4": (2, 2, 16)}


def _fmt4(fmt: str) -> int:
    if fmt not in ("mxfp4", "nvfp4"):
        raise ValueError(f"fmt must be 'mxfp4' or 'nvfp4', not {fmt!r}")
    return QFMT[fmt]


def _check_tensor_scale(fmt: str, g: torch.Tensor) -> None:
    if fmt != "nvfp4":
        raise ValueError(f"a tensor scale belongs to nvfp4, not {fmt}")
    if g.dtype != torch.float32 or g.numel() != 1 or not g.is_cuda:
        raise ValueError("the tensor scale must be one fp32 value on the CUDA device")


def _rows_of(x: torch.Tensor, K: int) -> int:
    return x.numel() // K if K else 0


def quantize_fp4(x: torch.Tensor, fmt: str = "mxfp4", *,
                 tensor_scale: torch.Tensor | None = None) -> tuple[torch.Tensor, torch.Tensor]:
    """bf16 x [..., K] -> (x_q uint8 [..., K/2], two E2M1 codes a byte, the even
    element in the low half; x_scale uint8: "mxfp4" E8M0 [..., K/32], "nvfp4"
    E4M3 [..., K/16]).  ``tensor_scale``: nvfp4's fp32 scale of the whole tensor
    (one element on the device, >= 0; None is 1), normally amax / (448 * 6): 0 for
    an all-zero tensor, whose values are then 0."""
    f = _fmt4(fmt)
    if x.dtype is not _BF16:
        raise TypeError("x must be bfloat16")
    if not (x.is_cuda and x.is_contiguous()):
        _require_cuda(x)
    if tensor_scale is not None:
        _check_tensor_scale(fmt, tensor_scale)
    if x.data_ptr() & 15:
        x = _aligned16(x)
    shape, dev = x.shape, x.device
    lead, K = shape[:-1], shape[-1]
    q = torch.empty(lead + (K // 2,), dtype=_U8, device=dev)
    s = torch.empty(lead + (K // QBLOCK[fmt],), dtype=_U8, device=dev)
    _check(load().mxfp8_fp4_quantize(f, x.data_ptr(), x.numel() // K if K else 0, K,
                                     None if tensor_scale is None else tensor_scale.data_ptr(), q.data_ptr(),
                                     s.data_ptr(), _stream()))
    return q, s


def unpack_fp4(x_q: torch.Tensor) -> torch.Tensor:
    """Packed E2M1 codes [..., K/2] -> the same values as float8_e4m3fn [..., K]
    (with the same scales an MXFP4 tensor is then an MXFP8 one)."""
    if x_q.dtype is not _U8:
        raise TypeError("codes must be uint8")
    if not (x_q.is_cuda and x_q.is_contiguous()):
        _require_cuda(x_q)
    src = x_q.data_ptr()
    if src & 15:
        x_q = _aligned16(x_q)
        src = x_q.data_ptr()
    shape = x_q.shape
    out = torch.empty(shape[:-1] + (2 * shape[-1],), dtype=_E4M3, device=x_q.device)
    _check(load().mxfp8_fp4_unpack(src, out.numel(), out.data_ptr(), _stream()))
    return out


@functools.lru_cache(maxsize=4096)
def packed_sizes_fp4(B: int, N: int, K: int, fmt: str) -> tuple[int, int]:
    wb, sb = ctypes.c_size_t(), ctypes.c_size_t()
    _check(load().mxfp8_fp4_packed_sizes(_fmt4(fmt), B, N, K, ctypes.byref(wb), ctypes.byref(sb)))
    return wb.value, sb.value


def process_weights_fp4(w_q: torch.Tensor, w_scale: torch.Tensor, fmt: str = "mxfp4", *,
                        tensor_scale: torch.Tensor | None = None) -> PackedWeights:
    """w_q uint8 [N, K/2] or [B, N, K/2], w_scale uint8 (or the scale's float8
    type) [..., K/32] ("mxfp4") or [..., K/16] ("nvfp4"), and nvfp4's fp32
    ``tensor_scale`` -> weights for linear_fp4.  Padded scales are sliced as in
    process_weights."""
    f = _fmt4(fmt)
    if w_q.dim() not in (2, 3) or w_q.dtype != torch.uint8:
        raise ValueError("w_q must be uint8 [N, K/2] or [B, N, K/2]")
    batched = w_q.dim() == 3
    B, N, K = (w_q.shape[0] if batched else 1), w_q.shape[-2], 2 * w_q.shape[-1]
    if K % BLOCK:
        raise ValueError(f"K={K} is not a multiple of {BLOCK}")
    KB = K // QBLOCK[fmt]
    if (w_scale.dim() != w_q.dim() or w_scale.element_size() != 1
            or tuple(w_scale.shape[:-2]) != tuple(w_q.shape[:-2])
            or w_scale.shape[-2] < N or w_scale.shape[-1] < KB):
        raise ValueError(f"weight scale {tuple(w_scale.shape)} does not match weight {tuple(w_q.shape)}")
    if tensor_scale is not None:
        _check_tensor_scale(fmt, tensor_scale)
    w_scale = _bytes(w_scale)[..., :N, :KB].contiguous()
    _require_cuda(w_q, w_scale)
    w_q, w_scale = _aligned16(w_q), _aligned16(w_scale)
    wb, sb = packed_sizes_fp4(B, N, K, fmt)
    wp = torch.empty(wb, dtype=torch.uint8, device=w_q.device)
    sp = torch.empty(sb, dtype=torch.uint8, device=w_q.device)
    _check(load().mxfp8_fp4_process_weights(f, _ptr(w_q), _ptr(w_scale), B, N, K, _ptr(wp), _ptr(sp), _stream()))
    return PackedWeights(wp, sp, B, N, K, batched, fmt, tensor_scale)


@functools.lru_cache(maxsize=4096)
def workspace_size_fp4(B: int, M: int, N: int, K: int, quantized: bool, fmt: str) -> int:
    n = ctypes.c_size_t()
    _check(load().mxfp8_fp4_workspace_size(_fmt4(fmt), B, M, N, K, int(quantized), ctypes.byref(n)))
    return n.value


@functools.lru_cache(maxsize=4096)
def product_workspace_fp4(B: int, M: int, N: int, K: int, fmt: str) -> int:
    """Bytes gemm_packed_fp4 needs to split K (0 where it does not)."""
    n = ctypes.c_size_t()
    _check(load().mxfp8_fp4_product_workspace_size(_fmt4(fmt), B, M, N, K, ctypes.byref(n)))
    return n.value


def _workspace(given: torch.Tensor | None, need: int, device) -> tuple[int | None, int, torch.Tensor | None]:
    """(pointer, bytes, the tensor to keep alive during the call)."""
    if given is None:
        if need == 0:
            return None, 0, None
        given = torch.empty(need, dtype=torch.uint8, device=device)
    return given.data_ptr(), given.numel() * given.element_size(), given


def _product_args(pw: PackedWeights, bias: torch.Tensor | None, out: torch.Tensor | None, rows: int) -> None:
    if bias is not None and (bias.dtype != torch.bfloat16 or tuple(bias.shape) != (pw.N,)):
        raise ValueError("bias must be bf16 [N]")
    if out is not None and (out.dtype != torch.bfloat16 or out.numel() != rows * pw.N):
        raise ValueError(f"out must be bf16 with {rows * pw.N} elements")


def linear_fp4(x: torch.Tensor, pw: PackedWeights, bias: torch.Tensor | None = None,
               x_scale: torch.Tensor | None = None, *, tensor_scale: torch.Tensor | None = None,
               out: torch.Tensor | None = None, workspace: torch.Tensor | None = None) -> torch.Tensor:
    """Linear layer with both operands in 4 bits (weights from
    process_weights_fp4).  ``x`` is bf16 [..., K] (quantised inside the call to
    the weights' format), or with ``x_scale`` the codes uint8 [..., K/2] of
    quantize_fp4; ``tensor_scale`` is nvfp4's scale of x either way.  For batched
    weights x is [B, M, ...].  Returns bf16 [..., N]."""
    # Most of the host's share of a small call is Python's: one pass, no helper
    # calls for what is absent or in order (same box, M = 1 11.5 -> 11.1 us, with
    # a workspace 18.2 -> 16.9)
    fmt, K, N, B = pw.fmt, pw.K, pw.N, pw.B
    f = _fmt4(fmt)
    quantized = x_scale is not None
    if not (x.is_cuda and x.is_contiguous()):
        _require_cuda(x)
    if x_scale is not None or out is not None or workspace is not None:
        _require_cuda(x_scale, out, workspace)
    g_ptr = b_ptr = s_ptr = None
    if tensor_scale is not None:
        _check_tensor_scale(fmt, tensor_scale)
        g_ptr = tensor_scale.data_ptr()
    if x.dtype is not (_U8 if quantized else _BF16):
        raise TypeError("x must be bfloat16, or uint8 codes with x_scale")
    shape = x.shape
    KX = K // 2 if quantized else K
    if not shape or shape[-1] != KX:
        raise ValueError(f"x {tuple(shape)} does not match weights with K={K}")
    if pw.batched and (len(shape) != 3 or shape[0] != B):
        raise ValueError("batched weights need x of shape [B, M, K]")
    lead = shape[:-1]
    rows = x.numel() // KX
    if bias is not None:
        if not (bias.is_cuda and bias.is_contiguous()):
            _require_cuda(bias)
        if bias.dtype is not _BF16 or bias.dim() != 1 or bias.shape[0] != N:
            raise ValueError("bias must be bf16 [N]")
        b_ptr = bias.data_ptr()
        if b_ptr & 15:
            bias = _aligned16(bias)
            b_ptr = bias.data_ptr()
    if quantized:
        if x_scale.element_size() != 1 or x_scale.shape != lead + (K // QBLOCK[fmt],):
            raise ValueError(f"{fmt} activation scale {tuple(x_scale.shape)} for codes {tuple(shape)}")
        x_scale = _aligned16(x_scale)
        s_ptr = x_scale.data_ptr()
    if out is None:
        out = torch.empty(lead + (N,), dtype=_BF16, device=x.device)
    elif out.dtype is not _BF16 or out.numel() != rows * N:
        raise ValueError(f"out must be bf16 with {rows * N} elements")
    if rows == 0:
        return out
    x_ptr = x.data_ptr()
    if x_ptr & 15:
        x = _aligned16(x)
        x_ptr = x.data_ptr()
    M = rows // B
    need = workspace_size_fp4(B, M, N, K, quantized, fmt)
    ws_ptr, ws_bytes = None, 0
    if workspace is not None or need:
        ws_ptr, ws_bytes, workspace = _workspace(workspace, need, x.device)
    wg = pw.tensor_scale
    _check(load().mxfp8_fp4_linear(f, None if quantized else x_ptr, x_ptr if quantized else None, s_ptr, g_ptr, B, M, N, K,
                                   pw.w_packed.data_ptr(), pw.sf_packed.data_ptr(),
                                   None if wg is None else wg.data_ptr(), b_ptr, out.data_ptr(), ws_ptr, ws_bytes,
                                   _stream()))
    return out


def quantize_packed_fp4(x: torch.Tensor, B: int = 1, fmt: str = "mxfp4", *,
                        tensor_scale: torch.Tensor | None = None) -> PackedActivation:
    """bf16 x ([M, K], or [B, M, K] with B given) -> codes and packed scales for gemm_packed_fp4."""
    f = _fmt4(fmt)
    if x.dtype != torch.bfloat16:
        raise TypeError("x must be bfloat16")
    _require_cuda(x)
    if tensor_scale is not None:
        _check_tensor_scale(fmt, tensor_scale)
    x = _aligned16(x)
    K = x.shape[-1]
    rows = _rows_of(x, K)
    if B < 1 or rows % B:
        raise ValueError(f"x {tuple(x.shape)} does not split into B={B} batches")
    pa = _packed_activation(B, rows // B, K, fmt, tensor_scale, x.device)
    _check(load().mxfp8_fp4_quantize_packed(f, _ptr(x), B, pa.M, K, _ptr(tensor_scale), _ptr(pa.x_q),
                                            _ptr(pa.sf_packed), _stream()))
    return pa


@functools.lru_cache(maxsize=4096)
def _packed_sizes_mx8(B: int, M: int, K: int, fmt: str) -> tuple[int, int]:
    return packed_sizes(B, M, K)


def _packed_activation(B: int, M: int, K: int, fmt: str, tensor_scale: torch.Tensor | None,
                       device) -> PackedActivation:
    sb = (_packed_sizes_mx8 if fmt == "mxfp8" else packed_sizes_fp4)(B, max(M, 1), K, fmt)[1]
    return PackedActivation(torch.empty((B, M, K if fmt == "mxfp8" else K // 2), dtype=torch.uint8, device=device),
                            torch.empty(sb, dtype=torch.uint8, device=device), B, M, K, fmt, tensor_scale)


def gemm_packed_fp4(pa: PackedActivation, pw: PackedWeights, bias: torch.Tensor | None = None,
                    out: torch.Tensor | None = None, *, workspace: torch.Tensor | None = None) -> torch.Tensor:
    """The 4-bit product alone (x quantised by quantize_packed_fp4,
    rmsnorm_quantize or silu_mul_quantize with packed scales); bf16 [B, M, N].
    ``workspace`` (product_workspace_fp4 bytes) is allocated when the call splits
    K and none is given."""
    f = _fmt4(pw.fmt)
    if pa.fmt != pw.fmt or pa.K != pw.K or pa.B != pw.B:
        raise ValueError("activation and weights disagree on format, K or B")
    _require_cuda(bias, out, workspace)
    _product_args(pw, bias, out, pa.B * pa.M)
    bias = _aligned16(bias)
    if out is None:
        out = torch.empty((pa.B, pa.M, pw.N), dtype=torch.bfloat16, device=pa.x_q.device)
    if pa.M == 0:
        return out
    ws_ptr, ws_bytes, workspace = _workspace(workspace, product_workspace_fp4(pa.B, pa.M, pw.N, pa.K, pw.fmt),
                                             pa.x_q.device)
    _check(load().mxfp8_fp4_gemm_packed(f, pa.x_q.data_ptr(), pa.sf_packed.data_ptr(), _ptr(pa.tensor_scale), pa.B,
                                        pa.M, pw.N, pa.K, pw.w_packed.data_ptr(), pw.sf_packed.data_ptr(),
                                        _ptr(pw.tensor_scale), _ptr(bias), out.data_ptr(), ws_ptr, ws_bytes,
                                        _stream()))
    return out


# ------------------------------------------------------------------ steps that feed a quantised layer
def _rows2d(x: torch.Tensor, name: str) -> tuple[torch.Tensor, int, int]:
    """x [..., K] as rows: (tensor, row count, row stride in elements).  A view
    whose rows are evenly spaced (a slice of a wider tensor) is taken as it is
    when its rows start on 16-byte boundaries; anything else is copied."""
    if not x.is_cuda:
        raise ValueError("tensors must be on a CUDA device")
    shape = x.shape
    K = shape[-1] if shape else 0
    if K == 0 or K % BLOCK:
        raise ValueError(f"{name} must be [..., K] with K a multiple of {BLOCK}, not {tuple(shape)}")
    rows = x.numel() // K
    if x.is_contiguous():
        return (x if x.data_ptr() % 16 == 0 else _aligned16(x)), rows, K
    stride, step = 0, 1  # of the merged leading axes
    for size, st in zip(reversed(x.shape[:-1]), reversed(x.stride()[:-1])):
        if size == 1:
            continue
        if step == 1:
            stride = st
        elif st != stride * step:
            step = -1
            break
        step *= size
    if (step < 0 or x.stride(-1) != 1 or x.data_ptr() % 16 or stride * x.element_size() % 16
            or (rows > 1 and stride < K)):
        return x.contiguous(), rows, K
    return x, rows, stride


def _quantized_out(lead, device, rows: int, K: int, fmt: str, tensor_scale: torch.Tensor | None, packed: bool):
    """Output tensors of a fused quantising step: (what the caller gets, codes, scales)."""
    if packed:
        pa = _packed_activation(1, rows, K, fmt, tensor_scale, device)
        return pa, pa.x_q, pa.sf_packed
    _, per, block = _QSPEC[fmt]
    q = torch.empty(lead + (K // per,), dtype=_U8, device=device)
    s = torch.empty(lead + (K // block,), dtype=_U8, device=device)
    return (q, s), q, s


def _qfmt(fmt: str) -> int:
    if fmt not in _QSPEC:
        raise ValueError(f"fmt must be one of {sorted(_QSPEC)}, not {fmt!r}")
    return _QSPEC[fmt][0]


def rmsnorm_quantize(x: torch.Tensor, weight: torch.Tensor, residual: torch.Tensor | None = None, *,
                     eps: float = 1e-6, fmt: str = "mxfp8", tensor_scale: torch.Tensor | None = None,
                     packed: bool = False, residual_out: torch.Tensor | None = None,
                     y: torch.Tensor | None = None):
    """Residual addition and RMS norm, output quantised for the next layer:
    t = x + residual, y = t / sqrt(mean(t^2) + eps) * weight (fp32 throughout).

    x bf16 [..., K], weight bf16 [K], residual bf16 or fp32 like x (or None).
    Returns (quantised y, t rounded to the residual's type or None).  The
    quantised y is (codes, row-major scales) as quantize / quantize_fp4 return
    them, or with ``packed`` a PackedActivation of one batch for gemm_packed /
    gemm_packed_fp4.  ``residual_out`` (dense; may be a dense ``residual``
    itself) receives t; ``y`` (dense bf16) receives the norm unquantised too."""
    f = _qfmt(fmt)
    if x.dtype is not _BF16 or weight.dtype is not _BF16:
        raise TypeError("x and weight must be bfloat16")
    if tensor_scale is not None:
        _check_tensor_scale(fmt, tensor_scale)
    if not (weight.is_cuda and weight.is_contiguous()):
        _require_cuda(weight)
    if residual_out is not None or y is not None:
        _require_cuda(residual_out, y)
    shape = x.shape
    xr, rows, x_stride = _rows2d(x, "x")
    K = shape[-1]
    if weight.dim() != 1 or weight.shape[0] != K:
        raise ValueError(f"weight must be [{K}], not {tuple(weight.shape)}")
    r_ptr, r_stride, r_f32, t_ptr = None, 0, False, None
    dev = x.device
    if residual is not None:
        rt = residual.dtype
        r_f32 = rt is _F32
        if not (r_f32 or rt is _BF16) or residual.shape != shape:
            raise ValueError("residual must be bf16 or fp32 with x's shape")
        rr, _, r_stride = _rows2d(residual, "residual")
        if residual_out is None:
            residual_out = torch.empty(shape, dtype=rt, device=dev)
        elif residual_out.dtype is not rt or residual_out.shape != shape:
            raise ValueError("residual_out must have the residual's type and shape")
        r_ptr, t_ptr = rr.data_ptr(), residual_out.data_ptr()
    elif residual_out is not None:
        raise ValueError("residual_out needs a residual")
    if y is not None and (y.dtype is not _BF16 or y.shape != shape):
        raise ValueError("y must be bf16 with x's shape")
    if weight.data_ptr() & 15:
        weight = _aligned16(weight)
    res, q, s = _quantized_out(shape[:-1], dev, rows, K, fmt, tensor_scale, packed)
    _check(load().mxfp8_rmsnorm_quantize(f, xr.data_ptr(), x_stride, r_ptr, r_stride, r_f32, t_ptr, weight.data_ptr(),
                                         eps, None if tensor_scale is None else tensor_scale.data_ptr(), rows, K,
                                         q.data_ptr(), s.data_ptr(), packed, None if y is None else y.data_ptr(),
                                         _stream()))
    return res, residual_out


def silu_mul_quantize(gate_up: torch.Tensor, up: torch.Tensor | None = None, *, fmt: str = "mxfp8",
                      tensor_scale: torch.Tensor | None = None, packed: bool = False):
    """silu(gate) * up with the output quantised for the next layer.

    ``gate_up`` bf16 [..., 2 K] holds gate then up along the last axis (a merged
    projection's output); or pass gate [..., K] and ``up`` [..., K].  Returns
    the quantised result as rmsnorm_quantize does."""
    f = _qfmt(fmt)
    if gate_up.dtype is not _BF16 or (up is not None and up.dtype is not _BF16):
        raise TypeError("gate and up must be bfloat16")
    if tensor_scale is not None:
        _check_tensor_scale(fmt, tensor_scale)
    if up is None:
        if gate_up.dim() < 1 or gate_up.shape[-1] % (2 * BLOCK):
            raise ValueError(f"gate_up must be [..., 2 K] with K a multiple of {BLOCK}, not {tuple(gate_up.shape)}")
        both, rows, stride = _rows2d(gate_up, "gate_up")
        K = gate_up.shape[-1] // 2
        lead = gate_up.shape[:-1]
        gate_ptr, gate_stride = both.data_ptr(), stride
        up_ptr, up_stride = gate_ptr + 2 * K, stride
    else:
        if up.shape != gate_up.shape:
            raise ValueError("gate and up must have the same shape")
        gr, rows, gate_stride = _rows2d(gate_up, "gate")
        ur, _, up_stride = _rows2d(up, "up")
        K, lead = gate_up.shape[-1], gate_up.shape[:-1]
        gate_ptr, up_ptr = gr.data_ptr(), ur.data_ptr()
    res, q, s = _quantized_out(lead, gate_up.device, rows, K, fmt, tensor_scale, packed)
    _check(load().mxfp8_silu_mul_quantize(f, gate_ptr, gate_stride, up_ptr, up_stride,
                                          None if tensor_scale is None else tensor_scale.data_ptr(), rows, K,
                                          q.data_ptr(), s.data_ptr(), packed, _stream()))
    return res


@functools.lru_cache(maxsize=4096)
def gated_mlp_workspace_size(fmt: str, M: int, K: int, F: int) -> int:
    n = ctypes.c_size_t()
    _check(load().mxfp8_gated_mlp_workspace_size(_qfmt(fmt), M, K, F, ctypes.byref(n)))
    return n.value


def gated_mlp(x: torch.Tensor, norm_weight: torch.Tensor, gate_up: PackedWeights, down: PackedWeights,
              residual: torch.Tensor | None = None, *, eps: float = 1e-6,
              x_tensor_scale: torch.Tensor | None = None, h_tensor_scale: torch.Tensor | None = None,
              workspace: torch.Tensor | None = None) -> tuple[torch.Tensor, torch.Tensor | None]:
    """A gated MLP block in one call (mxfp8_gated_mlp): rmsnorm_quantize of x (+
    residual), the gate_up product, silu_mul_quantize and the down product, all
    in the weights' format.  Returns (bf16 out like x, x + residual or None).
    x_tensor_scale / h_tensor_scale: nvfp4's scales of the norm's and the
    activation's output.  mlp.GatedMLP keeps the weights and checks them once."""
    fmt = "mxfp8" if gate_up.fmt == "e4m3" else gate_up.fmt
    f, K, F = _qfmt(fmt), gate_up.K, down.K
    if gate_up.fmt != down.fmt or gate_up.batched or down.batched or gate_up.N != 2 * F or down.N != K:
        raise ValueError(f"gate_up [{gate_up.N}, {K}] {gate_up.fmt} and down [{down.N}, {F}] {down.fmt} are not "
                         "[2 F, K] and [K, F] of one format")
    if x.dtype is not _BF16 or norm_weight.dtype is not _BF16:
        raise TypeError("x and norm_weight must be bfloat16")
    _require_cuda(norm_weight, workspace)
    for g in (x_tensor_scale, h_tensor_scale):
        if g is not None:
            _check_tensor_scale(fmt, g)
    shape, dev = x.shape, x.device
    xr, rows, x_stride = _rows2d(x, "x")
    if shape[-1] != K or tuple(norm_weight.shape) != (K,):
        raise ValueError(f"x {tuple(shape)} and norm_weight {tuple(norm_weight.shape)} do not match K={K}")
    r_ptr, r_stride, r_f32, t, t_ptr = None, 0, False, None, None
    if residual is not None:
        rt = residual.dtype
        r_f32 = rt is _F32
        if not (r_f32 or rt is _BF16) or residual.shape != shape:
            raise ValueError("residual must be bf16 or fp32 with x's shape")
        rr, _, r_stride = _rows2d(residual, "residual")
        t = torch.empty(shape, dtype=rt, device=dev)
        r_ptr, t_ptr = rr.data_ptr(), t.data_ptr()
    norm_weight = _aligned16(norm_weight)
    out = torch.empty(shape, dtype=_BF16, device=dev)
    ws_ptr, ws_bytes, workspace = _workspace(workspace, gated_mlp_workspace_size(fmt, rows, K, F), dev)
    _check(load().mxfp8_gated_mlp(f, xr.data_ptr(), x_stride, r_ptr, r_stride, r_f32, t_ptr, norm_weight.data_ptr(), eps,
                                  rows, K, F, gate_up.w_packed.data_ptr(), gate_up.sf_packed.data_ptr(),
                                  _ptr(gate_up.tensor_scale), down.w_packed.data_ptr(), down.sf_packed.data_ptr(),
                                  _ptr(down.tensor_scale), _ptr(x_tensor_scale), _ptr(h_tensor_scale), out.data_ptr(),
                                  ws_ptr, ws_bytes, _stream()))
    return out, t


def check() -> None:
    """Synchronise the current stream and raise if a kernel wait ran out."""
    _check(load().mxfp8_check(_stream()))


def debug_expire_wait(timeout_ns: int) -> None:
    _check(load().mxfp8_debug_expire_wait(timeout_ns, _stream()))
