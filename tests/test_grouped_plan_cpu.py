"""Which kernel and tile the shapes of _grouped_shapes are run by, asked of the library's own choice: a
change of that choice does not take a kernel's tests away unseen."""

import ctypes

import pytest

from _grouped_shapes import BATCHED, DENSE, GROUPED, GROUPED_RAGGED_K
from mxfp8_block_scaled_02_gb300 import build, ops

MX, B128 = 0, 1


class Plan(ctypes.Structure):
    _fields_ = [("cg", ctypes.c_int), ("tn", ctypes.c_int), ("splits", ctypes.c_int)]


@pytest.fixture(scope="module")
def plan():
    build.build()
    fn = ops.load()._ZN2mx12grouped_planEillllb  # mx::grouped_plan(int, int64_t x 4, bool)
    fn.restype, fn.argtypes = Plan, [ctypes.c_int] + [ctypes.c_int64] * 4 + [ctypes.c_bool]

    def ask(fmt, groups, rows, N, K, ragged):
        p = fn(fmt, groups, rows, N, K, ragged)
        return p.cg, p.tn, p.splits

    return ask


def test_dense(plan):
    for (M, N, K), want in DENSE:
        assert plan(B128, 1, M, N, K, False) == want, (M, N, K)
    for (B, M, N, K), want in BATCHED:
        assert plan(B128, B, B * M, N, K, False) == want, (B, M, N, K)
    assert {want for _, want in DENSE} == {(2, 256, 1), (1, 128, 1), (1, 64, 1), (1, 32, 1), (1, 16, 1)}


@pytest.mark.parametrize("fmt", [MX, B128])
def test_grouped(plan, fmt):
    for counts, N, K, want in GROUPED + (GROUPED_RAGGED_K if fmt == B128 else []):
        assert plan(fmt, len(counts), sum(counts), N, K, True) == want, (counts, N, K)
