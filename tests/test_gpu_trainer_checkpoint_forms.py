"""SwiGLUTrainer(checkpoint="fp8") with the other forms of the optimizer: the same bits
as with its default form over several steps."""
import pytest
import torch

from gpu_util import lib

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("form", [dict(fuse_optimizer=True), dict(overlap_optimizer=True)])
@pytest.mark.parametrize("scaling", ["delayed", "auto"])
def test_optimizer_forms(form, scaling):
    F = lib()
    from fp8_quantized_gemm_gb300.mlp import SwiGLUTrainer
    T, d, ffn = 272, 256, 528
    g = torch.Generator(device="cuda").manual_seed(1)
    w1, w3, w2 = ((torch.randn(s, generator=g, device="cuda") * 0.06).bfloat16() for s in ((ffn, d), (ffn, d), (d, ffn)))
    a, b = (SwiGLUTrainer(w1, w3, w2, T, history=4, checkpoint="fp8", weight_scaling=scaling, **f) for f in ({}, form))
    x = torch.randn((T, d), generator=g, device="cuda").bfloat16()
    for _ in range(4):
        dy = (torch.randn((T, d), generator=g, device="cuda") * 1e-2).bfloat16()
        a.step(x, dy)
        b.step(x, dy)
        torch.cuda.synchronize()
        for name in ("aq", "y", "da", "dhq", "duq", "dx", "scale"):
            assert torch.equal(getattr(a, name), getattr(b, name)), name
        for key in a.kept:
            assert torch.equal(a.kept[key], b.kept[key]), key
        for name in ("w_master", "m", "v"):
            for p, q in zip(getattr(a, name), getattr(b, name)):
                assert torch.equal(p, q), name
    assert F.fp8_get_last_device_error() == (0, 0)
