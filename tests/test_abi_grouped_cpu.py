"""The block-128, grouped, routing and expert calls without a GPU: sizes, and argument errors found
before any device is touched; the binding's own refusals."""

import ctypes

import pytest
import torch

from mxfp8_block_scaled_02_gb300 import build, mlp, ops

P = ctypes.c_void_p
FAKE = P(0x10000)  # never dereferenced: every call below fails its checks first
ODD = P(0x10008)
MX, B128 = 0, 1
INVALID, UNSUPPORTED = 1, 2


@pytest.fixture(scope="module")
def lib():
    build.build()
    return ops.load()


def caller(fn, ok):
    def call(**kw):
        a = list(ok)
        for i, v in kw.items():
            a[int(i[1:])] = v
        return fn(*a)
    return call


def test_sizes(lib):
    up = lambda v: -(-v // 256) * 256  # noqa: E731
    assert ops.workspace_size_fp8_128(2, 3, 128, 400, False) == up(6 * 400) + up(4 * 6 * 4)
    assert ops.workspace_size_fp8_128(1, 4096, 14336, 4096, False) == 4096 * 4096 + 4 * 4096 * 32
    assert ops.workspace_size_fp8_128(1, 4096, 14336, 4096, True) == 0
    # one to eight rows are quantised in the product's kernel
    assert ops.workspace_size_fp8_128(1, 8, 256, 512, False) == 0 and ops.workspace_size_fp8_128(1, 9, 256, 512, False) > 0
    assert ops.grouped_workspace_size("e4m3", 8, 100, 256, 512, False) == up(100 * 512) + up(4 * 100 * 4)
    assert ops.grouped_workspace_size("fp8_128", 8, 100, 256, 512, True) == 0
    assert ops.route_workspace_size(32, 128, 8) == 0          # one CTA
    assert ops.route_workspace_size(33, 128, 8) == ops.route_workspace_size(1 << 20, 128, 8) == 160 * 128 * 4
    assert ops.route_workspace_size(0, 8, 2) == 0
    assert ops.expert_mlp_workspace_size("fp8_128", 0, 8, 2, 256, 128) >= 0


def test_quantise_errors(lib):
    call = caller(lib.mxfp8_b128_quantize, [FAKE, 4, 64, FAKE, FAKE, None])
    assert call(_1=-1) == INVALID and call(_2=0) == INVALID
    assert call(_2=40) == UNSUPPORTED and call(_2=1 << 30) == UNSUPPORTED and call(_1=(1 << 30) + 1) == UNSUPPORTED
    assert call(_0=None) == INVALID and call(_3=ODD) == INVALID and call(_4=None) == INVALID
    assert call(_1=0, _0=None) == 0
    call = caller(lib.mxfp8_b128_quantize_weights, [FAKE, 2, 64, 64, FAKE, FAKE, None])
    assert call(_1=0) == INVALID and call(_2=0) == INVALID and call(_3=24) == UNSUPPORTED
    assert call(_0=ODD) == INVALID and call(_1=1 << 20, _2=1 << 29, _3=1 << 29) == UNSUPPORTED
    call = caller(lib.mxfp8_b128_silu_mul_quantize, [FAKE, 128, P(0x10080), 128, 4, 64, FAKE, FAKE, None])
    assert call(_1=60) == INVALID and call(_1=56) == INVALID and call(_3=132) == INVALID
    assert call(_2=None) == INVALID and call(_2=ODD) == INVALID and call(_6=None) == INVALID
    assert call(_5=24) == UNSUPPORTED and call(_4=0, _0=None) == 0


def test_linear_errors(lib):
    #       x     xq    xs    B  M  N    K    w     ws    bias  out   workspace  bytes stream
    ok = [FAKE, None, None, 1, 40, 256, 512, FAKE, FAKE, None, FAKE, P(0x10100), 1 << 20, None]
    call = caller(lib.mxfp8_b128_linear, ok)
    assert call(_3=0) == INVALID and call(_4=-1) == INVALID and call(_5=0) == INVALID and call(_6=0) == INVALID
    assert call(_5=12) == UNSUPPORTED and call(_6=520) == UNSUPPORTED
    assert call(_4=1 << 31) == INVALID and call(_3=1 << 21, _4=1) == UNSUPPORTED
    assert call(_4=1 << 30, _5=1 << 29) == UNSUPPORTED
    assert call(_1=FAKE) == INVALID and call(_0=None) == INVALID and call(_0=None, _1=FAKE) == INVALID
    assert call(_7=None) == INVALID and call(_8=ODD) == INVALID and call(_9=ODD) == INVALID and call(_10=None) == INVALID
    assert call(_11=None) == INVALID and call(_11=P(0x10010)) == INVALID and call(_12=100) == INVALID
    assert b"needs" in lib.mxfp8_last_error()
    assert call(_4=0, _0=None) == 0
    n = ctypes.c_size_t()
    assert lib.mxfp8_b128_workspace_size(1, 4, 256, 512, 0, None) == INVALID
    assert lib.mxfp8_b128_workspace_size(1, 4, 250, 512, 0, ctypes.byref(n)) == UNSUPPORTED


@pytest.mark.parametrize("fmt", [MX, B128])
def test_grouped_errors(lib, fmt):
    #      fmt  x     T   rows  xq    xs    offs  E  R  N    K    w     ws    bias  out   ws          bytes    stream
    ok = [fmt, FAKE, 4, FAKE, None, None, FAKE, 3, 6, 256, 512, FAKE, FAKE, None, FAKE, P(0x10100), 1 << 20, None]
    call = caller(lib.mxfp8_grouped_linear, ok)
    assert call(_0=2) == INVALID and call(_0=-1) == INVALID
    assert call(_3=None) == INVALID  # T rows, another number in the product
    assert call(_3=P(0x10002)) == INVALID and call(_6=None) == INVALID and call(_6=P(0x10001)) == INVALID
    assert call(_1=None, _4=FAKE, _5=FAKE) == INVALID  # rows with a quantised x
    assert call(_4=FAKE, _5=FAKE) == INVALID and call(_1=None, _3=None, _4=FAKE) == INVALID
    assert call(_7=0) == INVALID and call(_7=513) == UNSUPPORTED and call(_8=-1) == INVALID
    assert call(_9=20) == UNSUPPORTED and call(_10=(448 + 32 if fmt == MX else 520)) == UNSUPPORTED
    assert call(_8=1 << 31) == UNSUPPORTED and call(_8=1 << 30, _9=1 << 20) == UNSUPPORTED
    assert call(_2=-1) == INVALID and call(_11=None) == INVALID and call(_12=None) == INVALID and call(_13=ODD) == INVALID
    assert call(_14=ODD) == INVALID and call(_15=None) == INVALID and call(_16=64) == INVALID
    assert call(_8=0, _6=None) == 0


def test_route_errors(lib):
    #     logits str bf16 T  E   k  sc rn scale ids   w     offs  rows  pos   ws    bytes stream
    ok = [FAKE, 16, 0, 4, 16, 2, 0, 0, 1.0, FAKE, FAKE, FAKE, FAKE, FAKE, None, 0, None]
    call = caller(lib.mxfp8_route, ok)
    assert call(_3=-1) == INVALID and call(_4=0) == INVALID and call(_5=0) == INVALID and call(_5=17) == INVALID
    assert call(_4=513, _1=513) == UNSUPPORTED and call(_4=64, _5=33, _1=64) == UNSUPPORTED
    assert call(_3=1 << 30) == UNSUPPORTED and call(_6=2) == INVALID
    assert call(_1=15) == INVALID and call(_0=P(0x10002)) == INVALID and call(_0=None) == INVALID
    for i in (9, 10, 11, 12, 13):
        assert call(**{f"_{i}": None}) == INVALID
    assert call(_3=65) == INVALID and b"workspace" in lib.mxfp8_last_error()
    assert call(_3=65, _14=ODD, _15=1 << 20) == INVALID


def test_combine_errors(lib):
    ok = [FAKE, 8, FAKE, FAKE, 4, 2, 64, None, 0, FAKE, None]
    call = caller(lib.mxfp8_combine, ok)
    assert call(_1=-1) == INVALID and call(_4=-1) == INVALID and call(_5=0) == INVALID and call(_6=0) == INVALID
    assert call(_6=12) == UNSUPPORTED and call(_5=33) == UNSUPPORTED
    assert call(_0=None) == INVALID and call(_2=None) == INVALID and call(_9=ODD) == INVALID
    assert call(_7=ODD, _8=64) == INVALID and call(_7=FAKE, _8=56) == INVALID and call(_7=FAKE, _8=68) == INVALID
    assert call(_4=0, _9=None) == 0


def test_expert_mlp_errors(lib):
    #      fmt x    T  K    logit st bf E  k  sc rn scale F    gu    gus   dn    dns   add  st out   ws          bytes    stream
    ok = [B128, FAKE, 4, 256, FAKE, 8, 0, 8, 2, 0, 0, 1.0, 128, FAKE, FAKE, FAKE, FAKE, None, 0, FAKE, P(0x10100), 1 << 24, None]
    call = caller(lib.mxfp8_expert_mlp, ok)
    assert call(_0=2) == INVALID and call(_8=9) == INVALID and call(_9=3) == INVALID and call(_12=0) == INVALID
    assert call(_12=24) == UNSUPPORTED and call(_0=MX, _12=192) == UNSUPPORTED and call(_3=260) == UNSUPPORTED
    assert call(_7=600, _5=600) == UNSUPPORTED
    for i in (1, 4, 13, 14, 15, 16, 19):
        assert call(**{f"_{i}": None}) == INVALID
    assert call(_13=ODD) == INVALID and call(_17=FAKE, _18=100) == INVALID and call(_5=7) == INVALID
    assert call(_20=None) == INVALID and call(_20=P(0x10010)) == INVALID and call(_21=1024) == INVALID
    assert call(_2=0) == 0


def fake_weights(fmt, B, N, K, batched=True):
    return ops.PackedWeights(torch.empty(0, dtype=torch.uint8), torch.empty(0, dtype=torch.uint8), B, N, K, batched, fmt)


def test_binding_refusals(lib):
    bf, f32 = torch.bfloat16, torch.float32
    x = torch.empty(4, 256, dtype=bf)
    pw = fake_weights("fp8_128", 3, 128, 256)
    with pytest.raises(ValueError, match="CUDA"):
        ops.quantize_fp8_128(x)
    with pytest.raises(TypeError):
        ops.quantize_fp8_128(x.float())
    with pytest.raises(TypeError):
        ops.process_weights_fp8_128(torch.empty(128, 256, dtype=torch.uint8), torch.empty(1, 2, dtype=bf))
    with pytest.raises(ValueError, match="does not match"):
        ops.process_weights_fp8_128(torch.empty(129 + 7, 256, dtype=torch.uint8), torch.empty(1, 2, dtype=f32))
    with pytest.raises(ValueError, match="multiple"):
        ops.process_weights_fp8_128(torch.empty(128, 250, dtype=torch.uint8), torch.empty(1, 2, dtype=f32))
    with pytest.raises(ValueError, match="e4m3 weights"):
        ops.linear_fp8_128(x, fake_weights("e4m3", 1, 128, 256))
    with pytest.raises(TypeError):
        ops.linear_fp8_128(x.float(), pw)
    with pytest.raises(ValueError, match="linear_fp8_128"):
        ops.linear(x, pw)
    with pytest.raises(ValueError, match="linear_fp8_128"):
        ops.linear_noalloc(x, pw)
    with pytest.raises(ValueError, match="mxfp4"):
        ops.grouped_linear(x, fake_weights("mxfp4", 3, 128, 256), torch.zeros(4, dtype=torch.int32))
    with pytest.raises(ValueError, match="one matrix an expert"):
        ops.grouped_linear(x, fake_weights("e4m3", 1, 128, 256, False), torch.zeros(2, dtype=torch.int32))
    with pytest.raises(ValueError, match="rows go with"):
        ops.grouped_linear(x, pw, torch.zeros(4, dtype=torch.int32), x, rows=torch.zeros(4, dtype=torch.int32))
    with pytest.raises(ValueError, match="scoring"):
        ops.route(torch.zeros(2, 4), 1, scoring="max")
    with pytest.raises(ValueError, match="CUDA"):
        ops.route(torch.zeros(2, 4), 1)
    with pytest.raises(ValueError, match="packed"):
        ops.silu_mul_quantize(x, fmt="fp8_128", packed=True)
    with pytest.raises(ValueError, match="tensor scale"):
        ops.silu_mul_quantize(x, fmt="fp8_128", tensor_scale=torch.ones(1))
    with pytest.raises(ValueError, match="fmt must be"):
        ops.rmsnorm_quantize(x, x[0], fmt="fp8_128")
    with pytest.raises(ops.MxStatusError, match="experts=600"):
        ops.route_workspace_size(4, 600, 2)


def test_expert_mlp_refusals():
    gu, dn = fake_weights("fp8_128", 8, 512, 128), fake_weights("fp8_128", 8, 128, 256)
    mlp.ExpertMLP(gu, dn, 2)
    for bad in ((fake_weights("e4m3", 8, 512, 128), dn), (gu, fake_weights("fp8_128", 7, 128, 256)),
                (gu, fake_weights("fp8_128", 8, 128, 128)), (fake_weights("mxfp4", 8, 512, 128), fake_weights("mxfp4", 8, 128, 256)),
                (fake_weights("fp8_128", 1, 512, 128, False), fake_weights("fp8_128", 1, 128, 256, False))):
        with pytest.raises(ValueError):
            mlp.ExpertMLP(*bad, 2)
    with pytest.raises(ValueError, match="top_k"):
        mlp.ExpertMLP(gu, dn, 9)
    with pytest.raises(ValueError, match="scoring"):
        mlp.ExpertMLP(gu, dn, 2, scoring="max")
