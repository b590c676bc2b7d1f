"""Kernels that hold tensor memory let their dependents start only once they hold it.

A dependent that allocates tensor memory may share an SM with a CTA whose own
allocation is pending: if it is served first, it waits for this grid to finish
and this grid's allocation waits for its columns.  No run can show the order
safely, so the sources are read: in each kernel the allocation, then a barrier of
the CTA, then the trigger."""

import glob
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "bit_weight_only_gemv_gb300", "csrc")


def code(path):
    with open(path) as f:
        return re.sub(r"//[^\n]*|/\*.*?\*/", "", f.read(), flags=re.S)


HOLDERS = sorted(p for p in glob.glob(os.path.join(CSRC, "*.cu")) if "tcgen05.alloc" in code(p))


def test_there_are_such_kernels():
    assert len(HOLDERS) >= 4


@pytest.mark.parametrize("path", HOLDERS, ids=[os.path.basename(p) for p in HOLDERS])
def test_trigger_comes_after_the_allocation(path):
    kernels = [k for k in re.split(r"\b__global__\b", code(path))[1:] if "tcgen05.alloc" in k]
    assert kernels
    for k in kernels:
        alloc = k.index("tcgen05.alloc")
        barrier = k.index("__syncthreads", alloc)
        triggers = [m.start() for m in re.finditer(r"pdl_launch_dependents\(\)", k)]
        # (a kernel that follows in the same file has its own trigger, after its own braces)
        assert triggers and triggers[0] > barrier
