"""Device memory that the library touches on the host's behalf is touched in
the order of the caller's stream (host only: the sources).  cudaMemset and
cudaMemcpy without a stream run on the legacy default stream, which streams
created as non-blocking (torch's are) do not wait for: a buffer cleared that
way may be cleared after the first kernel has filled it."""
import os
import re

import fp8_quantized_gemm_gb300 as F

CSRC = os.path.join(os.path.dirname(F.__file__), "csrc")


def calls(name):
    for f in sorted(os.listdir(CSRC)):
        with open(os.path.join(CSRC, f)) as h:
            s = re.sub(r"//[^\n]*", "", h.read())
        for m in re.finditer(r"\b%s\s*\(" % name, s):
            yield f, s[:m.start()].count("\n")


def test_no_memset_outside_the_stream():
    assert not list(calls("cudaMemset"))


def test_no_copy_outside_the_stream():
    """The device error word alone is read that way, behind a synchronize."""
    assert {f for f, _ in calls("cudaMemcpy")} <= {"api.cu"}
    assert len(list(calls("cudaMemcpy"))) == 2
