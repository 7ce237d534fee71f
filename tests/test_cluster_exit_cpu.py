"""Signals to another CTA's barriers and the end of the kernel, by the text of the sources.

A CTA's shared memory must not be signalled once it has left.  Arrivals on another CTA's barrier that
this CTA does not wait for before it leaves are ordered by the cluster barrier at the end alone, and
only by its releasing form."""

import glob
import os
import re

import pytest

from mxfp8_block_scaled_02_gb300 import build

SIGNAL = "mbar_arrive_remote("


def kernels_that_signal() -> dict:
    found = {}
    for path in sorted(glob.glob(os.path.join(build.CSRC, "*.cu"))):
        with open(path) as f:
            text = re.sub(r"//[^\n]*", "", f.read())
        if SIGNAL in text:
            found[os.path.basename(path)] = text
    return found


@pytest.mark.parametrize("name", sorted(kernels_that_signal()))
def test_the_last_cluster_barrier_orders_the_signals(name):
    text = kernels_that_signal()[name]
    end = text[text.rindex(SIGNAL):]
    end = end[:end.index("tmem_dealloc_pair")]
    last = max(end.rfind("cluster_arrive_relaxed();"), end.rfind("cluster_sync();"))
    assert last >= 0, "no cluster barrier before the end"
    # on pairs (the kernels that signal): a releasing barrier
    pairs = re.search(r"if \(CG == 2\)\s*\{?\s*cluster_sync\(\);", end)
    assert pairs or end.startswith("cluster_sync();", last), "the barrier before the end orders no signal"


def test_some_kernels_signal():
    assert {"gemm_b128_pair.cu", "gemm_grouped.cu", "gemm_pair.cu", "gemm_fp4.cu"} <= set(kernels_that_signal())


def test_a_wait_that_ran_out_still_waits_for_what_others_send():
    """The grouped product's K splits: no partial sum may land after the CTA that it was sent to has left."""
    with open(os.path.join(build.CSRC, "gemm_grouped.cu")) as f:
        text = re.sub(r"//[^\n]*", "", f.read())
    epilogue = text[text.index("auto finish_split ="):]
    epilogue = epilogue[epilogue.index("const bool split"):epilogue.index("__syncthreads();")]
    for leave in re.finditer(r"\bbreak;", epilogue):
        before = epilogue[:leave.start()].rstrip()
        assert before.endswith("finish_split();"), before[-200:]
