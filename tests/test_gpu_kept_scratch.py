"""The kept scratch on the device: a refused call leaves nothing behind, and
streams that are not torch's own get right results."""
import ctypes

import pytest
import torch

from gpu_util import lib

pytestmark = pytest.mark.gpu


def test_backward_on_streams_of_all_kinds():
    F = lib()
    m, k = 700, 1040
    g = torch.Generator(device="cuda").manual_seed(0)
    dy, r = (torch.randn(m, k, generator=g, device="cuda") for _ in range(2))
    inv = torch.rsqrt(r.square().mean(1) + 1e-5)
    ws = torch.empty(F.fp8_rmsnorm_backward_workspace(m, k), dtype=torch.uint8, device="cuda")
    want, dx = torch.empty(k, device="cuda"), torch.empty_like(r)
    F.fp8_rmsnorm_backward(dy, r, inv, None, dx, dw=want, workspace=ws)
    with pytest.raises(ValueError):
        F.fp8_rmsnorm_backward(dy, r, inv[:-1], None, dx, dw=torch.empty_like(want))
    rt, raw = ctypes.CDLL("libcudart.so.13"), []
    for _ in range(2):
        h = ctypes.c_void_p()
        assert rt.cudaStreamCreateWithFlags(ctypes.byref(h), 1) == 0
        raw.append(torch.cuda.ExternalStream(h.value))
    streams = [torch.cuda.default_stream(), torch.cuda.Stream(), torch.cuda.Stream(priority=-1)] + raw
    torch.cuda.synchronize()
    got = []
    for _ in range(5):
        for st in streams:
            with torch.cuda.stream(st):
                dw, d = torch.empty_like(want), torch.empty_like(r)
                F.fp8_rmsnorm_backward(dy, r, inv, None, d, dw=dw)
                got += [(dw, d)]
    torch.cuda.synchronize()
    assert all(torch.equal(a, want) and torch.equal(b, dx) for a, b in got)
    kept = {sid for _, sid in F._kept.buffers}
    assert not kept & {st.cuda_stream for st in raw} and 0 in kept
    assert len(kept) >= 3  # the default stream and torch's two
