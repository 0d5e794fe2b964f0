"""The package imports, and its host-side checks answer, on a torch that lacks
the accessors of its CUDA build (host only; in a child process)."""
import os
import subprocess
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

CHILD = """
import torch
for name in [n for n in dir(torch._C) if n.startswith("_cuda_")]:
    delattr(torch._C, name)
import fp8_quantized_gemm_gb300 as F
x = torch.zeros(4, 32)
for call in (lambda: F.fp8_rmsnorm_quantize(x, None, 1e-5, F.E4M3, x, scale=x),
             lambda: F.fp8_gemm_tensor_act_backward(x, 0, x, 0, x, x, x, F.ACT_RELU, out=x)):
    try:
        call()
    except ValueError:
        continue
    raise SystemExit("a CPU tensor was taken")
print("imported", F.fp8_rmsnorm_backward_workspace(8, 256) > 0)
"""


def test_import():
    p = subprocess.run([sys.executable, "-c", CHILD], cwd=ROOT, capture_output=True, text=True,
                       timeout=300)
    assert p.returncode == 0 and p.stdout.split() == ["imported", "True"], p.stderr[-2000:]
