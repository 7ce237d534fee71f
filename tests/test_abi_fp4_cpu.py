"""The 4-bit, norm and activation calls of the C ABI without a GPU: sizes, and argument errors found before any
device is touched."""

import ctypes

import pytest
import torch  # noqa: F401  (loads the CUDA runtime the library links against)

from mxfp8_block_scaled_02_gb300 import build, ops

P = ctypes.c_void_p
FAKE = P(0x10000)  # never dereferenced: every call below fails its checks first
MX8, MX4, NV4 = 0, 1, 2


@pytest.fixture(scope="module")
def lib():
    build.build()
    return ops.load()


def test_sizes(lib):
    assert ops.packed_sizes_fp4(1, 256, 512, "mxfp4") == (256 * 256, 2 * 4 * 512)
    assert ops.packed_sizes_fp4(1, 256, 512, "nvfp4") == (256 * 256, 2 * 8 * 512)
    # ragged rows and K round up to whole atoms (128 rows x 128 or 64 elements)
    assert ops.packed_sizes_fp4(2, 129, 160, "mxfp4") == (2 * 129 * 80, 2 * 2 * 2 * 512)
    assert ops.packed_sizes_fp4(2, 129, 160, "nvfp4") == (2 * 129 * 80, 2 * 2 * 3 * 512)
    # one token is quantised in the product's kernel; codes need room for their repacked scales
    assert ops.workspace_size_fp4(1, 1, 4096, 4096, False, "mxfp4") == 0
    assert ops.workspace_size_fp4(1, 1, 4096, 4096, True, "mxfp4") == 32 * 512
    # many rows: codes and scales; no K split
    assert ops.workspace_size_fp4(1, 4096, 14336, 4096, False, "nvfp4") == 4096 * 2048 + 32 * 64 * 512
    assert ops.product_workspace_fp4(1, 4096, 14336, 4096, "nvfp4") == 0
    # few tiles and a long K: fp32 partials
    assert ops.product_workspace_fp4(1, 256, 1024, 28672, "mxfp4") == 8 * 4 * 256 * 1024
    # split in two within a cluster: none
    assert ops.product_workspace_fp4(1, 256, 4096, 14336, "mxfp4") == 0


def test_quantise_errors(lib):
    ok = [MX4, FAKE, 4, 64, None, FAKE, FAKE, None]

    def call(**kw):
        a = list(ok)
        for i, v in kw.items():
            a[int(i[1:])] = v
        return lib.mxfp8_fp4_quantize(*a)

    assert call(_0=MX8) == 1 and call(_0=7) == 1       # not a 4-bit format
    assert call(_2=-1) == 1 and call(_3=48) == 1 and call(_3=0) == 1
    assert call(_1=None) == 1 and call(_5=None) == 1 and call(_6=P(0x10004)) == 1
    assert call(_4=FAKE) == 1 and b"NVFP4" in lib.mxfp8_last_error()   # MXFP4 has no tensor scale
    assert call(_0=NV4, _4=P(0x10002)) == 1
    assert call(_2=1 << 31, _3=1 << 20) == 2           # more than 2^31 - 1 blocks
    assert call(_2=0) == 0                             # nothing to do
    assert lib.mxfp8_fp4_unpack(FAKE, 33, FAKE, None) == 1
    assert lib.mxfp8_fp4_unpack(None, 32, FAKE, None) == 1
    assert lib.mxfp8_fp4_unpack(P(0x10008), 32, FAKE, None) == 1
    assert lib.mxfp8_fp4_unpack(None, 0, None, None) == 0


def test_product_errors(lib):
    # fmt, x, x_q, x_scale, x_ts, B, M, N, K, w, sf, w_ts, bias, out, ws, ws_bytes, stream
    ok = [MX4, FAKE, None, None, None, 1, 64, 256, 512, FAKE, FAKE, None, None, FAKE, FAKE, 1 << 30, None]

    def call(**kw):
        a = list(ok)
        for i, v in kw.items():
            a[int(i[1:])] = v
        return lib.mxfp8_fp4_linear(*a)

    assert call(_0=MX8) == 1
    assert call(_2=FAKE, _3=FAKE) == 1 and b"exactly one" in lib.mxfp8_last_error()
    assert call(_1=None) == 1 and call(_1=None, _2=FAKE) == 1
    assert call(_5=0) == 1 and call(_6=-1) == 1 and call(_7=0) == 1 and call(_8=500) == 1
    assert call(_7=250) == 2 and b"N % 8" in lib.mxfp8_last_error()
    assert call(_9=None) == 1 and call(_10=None) == 1 and call(_13=None) == 1
    assert call(_1=P(0x10004)) == 1 and call(_13=P(0x10002)) == 1 and call(_12=P(0x10002)) == 1
    assert call(_4=FAKE) == 1 and call(_11=FAKE) == 1   # tensor scales are NVFP4's
    assert call(_15=16) == 1 and b"workspace" in lib.mxfp8_last_error()
    assert call(_14=P(0x10010)) == 1
    assert call(_5=1 << 19, _6=1 << 11, _7=1 << 20, _8=32) == 2
    assert call(_6=0, _1=None, _2=FAKE, _3=FAKE, _9=FAKE) == 0


def test_norm_and_activation_errors(lib):
    # fmt, x, x_stride, res, r_stride, r_f32, r_out, w, eps, ts, M, K, q, scale, packed, y, stream
    ok = [MX8, FAKE, 64, FAKE, 64, 0, FAKE, FAKE, 1e-6, None, 2, 64, FAKE, FAKE, 0, None, None]

    def norm(**kw):
        a = list(ok)
        for i, v in kw.items():
            a[int(i[1:])] = v
        return lib.mxfp8_rmsnorm_quantize(*a)

    assert norm(_0=3) == 1 and norm(_11=40) == 1 and norm(_11=32768 + 32) == 2
    assert norm(_8=-1.0) == 1 and norm(_8=float("nan")) == 1
    assert norm(_3=None) == 1 and norm(_6=None) == 1     # residual and residual_out go together
    assert norm(_2=60) == 1 and norm(_2=32) == 1 and norm(_4=68) == 1 and norm(_2=-64) == 1
    assert norm(_1=P(0x10008)) == 1 and norm(_7=None) == 1 and norm(_12=None) == 1 and norm(_13=P(0x10004)) == 1
    assert norm(_15=P(0x10002)) == 1 and norm(_9=FAKE) == 1
    assert norm(_10=0, _1=None) == 0
    # fmt, gate, g_stride, up, u_stride, ts, M, K, q, scale, packed, stream
    act_ok = [NV4, FAKE, 128, FAKE, 128, None, 2, 64, FAKE, FAKE, 1, None]

    def act(**kw):
        a = list(act_ok)
        for i, v in kw.items():
            a[int(i[1:])] = v
        return lib.mxfp8_silu_mul_quantize(*a)

    assert act(_0=-1) == 1 and act(_7=48) == 1 and act(_6=-1) == 1
    assert act(_1=None) == 1 and act(_3=None) == 1 and act(_3=P(0x10008)) == 1 and act(_2=36) == 1
    assert act(_8=None) == 1 and act(_9=P(0x10001)) == 1 and act(_5=P(0x10002)) == 1
    assert act(_6=0) == 0


def test_binding_refuses_formats_before_the_library():
    for f in ("mxfp8", "e2m1", "fp4"):
        with pytest.raises(ValueError):
            ops.packed_sizes_fp4(1, 8, 32, f)
    with pytest.raises(ValueError):
        ops.silu_mul_quantize(torch.zeros(2, 64, dtype=torch.bfloat16))  # not on a CUDA device
    with pytest.raises(ValueError):
        ops.rmsnorm_quantize(torch.zeros(2, 64, dtype=torch.bfloat16), torch.zeros(64, dtype=torch.bfloat16))
