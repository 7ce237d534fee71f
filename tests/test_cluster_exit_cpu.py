"""Signals to another CTA's barriers and the end of the kernel, by the text of the sources.

A CTA's shared memory must not be signalled once it has left.  So either the cluster barrier before the end
is the releasing one, which orders every signal ahead of it, or the CTA that is signalled has waited for the
last of them (and the barrier has a fence for a kernel in which a wait ran out)."""

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
    halves = [m.group() for m in re.finditer(r"cluster_sync\(\);|cluster_arrive_\w+\([^;]*\);", end)]
    assert halves, "no cluster barrier before the end"
    if re.search(r"if \(CG == 2\)\s*\{?\s*cluster_sync\(\);", end) or halves[-1] == "cluster_sync();":
        return  # releasing, on pairs at least (the kernels that signal)
    assert halves[-1] == "cluster_arrive_last(*abort_flag);", "the barrier before the end orders no signal"
    issuer = text[text.rindex("commit_pair_elected(elected, acc_full"):]
    issuer = issuer[:issuer.index("__nanosleep")]
    assert re.search(r"if \(ok &&[^;]*mbar_wait_warp\(acc_free,", issuer), "the last signals are not waited for"


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
