"""Kernels that start as programmatic dependents read what earlier kernels write through coherent loads.

A non-coherent load (__ldg, or a plain load through a const __restrict__ pointer) is not ordered by
griddepcontrol.wait: the compiler may take it to the kernel's start, while the kernel that writes the value
still runs.  No run can show that none is, so the sources are read: such loads are left for weights
alone, which a call's contract says that nothing still running writes."""

import glob
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "bit_weight_only_gemv_gb300", "csrc")
SOURCES = sorted(glob.glob(os.path.join(CSRC, "*.cu")) + glob.glob(os.path.join(CSRC, "*.cuh")))

# packed codes, steps and the experts' output vectors; the packers are plain launches (tested below)
WEIGHTS = {"gather.cu": ("qw", "st"), "gemv.cu": ("ov.s", "ov.b"), "quant.cu": ("codes", "w")}


def code(path):
    with open(path) as f:
        return re.sub(r"//[^\n]*|/\*.*?\*/", "", f.read(), flags=re.S)


def names(path):
    return os.path.basename(path)


@pytest.mark.parametrize("path", SOURCES, ids=names)
def test_non_coherent_loads_are_of_weights(path):
    text, allowed = code(path), WEIGHTS.get(os.path.basename(path), ())
    assert "ld.global.nc" not in text
    for m in re.finditer(r"__ldg\s*\((?:\s*reinterpret_cast<[^>]*>\()?\s*([\w.]+)", text):
        assert m.group(1) in allowed, f"__ldg({m.group(1)} ...)"
    for m in re.finditer(r"const\s+\w+\s*\*\s*__restrict__\s+(\w+)", text):
        assert m.group(1) in allowed, f"const __restrict__ {m.group(1)}"


def test_the_packers_are_plain_launches():
    text = code(os.path.join(CSRC, "quant.cu"))
    assert text.count("<<<") == 2 and "cudaLaunchKernelEx" not in text and "launch(" not in text
