"""Two pre-norm blocks in a chain, the lower one starting from the codes that the
upper one's norm gradient has written, over steps whose gradients shrink (with
a history of one step every scale follows).  Tolerances as in test_gpu_block.py:
twice the rms of the roundings on the way."""
import pytest
import torch

from gpu_util import lib
from test_gpu_block import make, plain, rel

pytestmark = pytest.mark.gpu


def grads64(x, s, dout, params):
    leaves = [v.double().requires_grad_() for v in (x, s) + params]
    r, branch = plain(*leaves)
    (branch + r + (r.bfloat16().double() - r).detach()).backward(dout.double())
    return [v.grad for v in leaves]


def test_chain():
    F = lib()
    from fp8_quantized_gemm_gb300 import block as B
    tokens, d, ffn = 160, 256, 528
    blocks = []
    for seed in (0, 1):
        w1, b1, w2, gain, rn = make(d, ffn, seed)
        t = B.PreNormMLPTrainer(w1, b1, w2, gain, tokens, history=1, lr=0.0, weight_decay=0.0)
        blocks.append((t, (w1, b1, w2, gain), rn(tokens, d).bfloat16(), rn(tokens, d, std=2.0).bfloat16()))
    (top, ptop, x1, s1), (low, plow, x0, s0) = blocks
    for i in range(5):
        dout = rn(tokens, d, std=0.5 * 8.0 ** -i).bfloat16()
        top.step(x1, dout, s1)
        live = top.scale[B.DR].item()
        low.step(x0, top.dr, s0, doutq=top.drq, dout_scale=top.drq_scale)
        if i < 2:  # the scales start from one
            continue
        assert live < 0.5 * top.drq_scale.item()  # update() has moved it on
        v = top.drq.view(torch.float8_e5m2).double() * top.drq_scale.double()
        assert rel(v, top.dr.double()) < 0.106
        for t, p, x, s, g in ((top, ptop, x1, s1, dout), (low, plow, x0, s0, top.dr)):
            gx, _, gw1, gb1, gw2, gg = grads64(x, s, g, p)
            assert rel(t.grads[0], gw1) < 0.174 and rel(t.grads[1], gw2) < 0.174
            assert rel(t.grads[2], gg) < 0.174 and rel(t.grads[3], gb1) < 0.174
            assert rel(t.dr.double() - g.double(), gx - g.double()) < 0.174
    with pytest.raises(ValueError):
        low.backward(top.dr, doutq=top.drq)
    assert F.fp8_get_last_device_error() == (0, 0)
