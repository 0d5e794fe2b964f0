"""Kernels launched with programmatic stream serialization start while the
kernel before them may still be writing their operands.  The read-only data
path (__ldg, or const __restrict__ pointers) is for data that is constant over
a kernel's lifetime, so none of them may use it (host only: the sources)."""
import os
import re

import pytest

import fp8_quantized_gemm_gb300 as F

CSRC = os.path.join(os.path.dirname(F.__file__), "csrc")
ATTR = "cudaLaunchAttributeProgrammaticStreamSerialization"


def source(name):
    with open(os.path.join(CSRC, name)) as f:
        return re.sub(r"//[^\n]*", "", f.read())


# the sources of these kernels and of what their epilogues call
WHOLE = ["gemm_skinny.cu", "gemm_kernel.cuh", "gemm_pair.cu", "gemm_common.cuh",
         "linear_epilogue.cuh", "activation.cuh", "pairs.cuh", "expert_tiles.cuh", "norm.cu"]


@pytest.mark.parametrize("name", WHOLE)
def test_no_read_only_loads(name):
    s = source(name)
    assert "__ldg" not in s and "ld.global.nc" not in s
    assert not re.search(r"const\s+[\w:]+\s*\*\s*__restrict__", s)


def test_group_quantizer_takes_unrestricted_input():
    """quantize.cu holds plainly launched kernels too: only the one that is
    launched programmatically is bound."""
    s = source("quantize.cu")
    at = s.index("quant_group_kernel(")
    head = s[at:s.index("{", at)]
    assert "__restrict__" not in head
    body = s[at:s.index("__global__", at)]
    assert "__ldg" not in body and "launch_dependents()" in body


def test_every_programmatic_launch_is_covered():
    """A file that starts to launch this way has to join the list above."""
    files = [f for f in os.listdir(CSRC) if f.endswith((".cu", ".cuh")) and ATTR in source(f)]
    assert set(files) <= set(WHOLE) | {"quantize.cu"}
