"""The pre-norm feed-forward block (block.py) against the same block in 64 bits
without quantization (plain torch, autograd for the gradients).

Tolerances.  One E4M3 rounding is a relative error of at most 2^-4 and about
2.6% rms, one E5M2 rounding 5.3% rms; a product of two independently rounded
operands accumulates them as noise.  The output goes through four E4M3
operands: 2.6% x sqrt(4) = 5.2% of the branch; a gradient through at most
three E4M3 and two E5M2 operands: sqrt(3 x 2.6^2 + 2 x 5.3^2) = 8.7%.  Both are
tested at twice that, the relative 2-norm of the difference.
"""
import pytest
import torch

from gpu_util import lib

pytestmark = pytest.mark.gpu


def rel(a, b):
    return ((a.double() - b).norm() / b.norm()).item()


def make(d, ffn, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rn = lambda *s, std=1.0: torch.randn(*s, generator=g, device="cuda") * std  # noqa: E731
    return rn(ffn, d, std=d ** -0.5), rn(ffn, std=0.3), rn(d, ffn, std=ffn ** -0.5), \
        1 + 0.1 * rn(d), rn


def plain(x, s, w1, b1, w2, gain, eps=1e-5):
    r = x + s
    y = r / torch.sqrt(r.square().mean(1, keepdim=True) + eps) * gain
    z = y @ w1.t() + b1
    a = torch.nn.functional.gelu(z, approximate="tanh")
    return r, a @ w2.t()


@pytest.mark.parametrize("tokens,d,ffn", [(96, 256, 528), (1000, 512, 2048)])
def test_training_step(tokens, d, ffn):
    F = lib()
    from fp8_quantized_gemm_gb300 import block as B
    w1, b1, w2, gain, rn = make(d, ffn)
    x, s = rn(tokens, d).bfloat16(), rn(tokens, d, std=2.0).bfloat16()
    dout = rn(tokens, d, std=1e-3).bfloat16()
    t = B.PreNormMLPTrainer(w1, b1, w2, gain, tokens, lr=0.0, weight_decay=0.0)
    for _ in range(3):  # the histories settle: from unit scales to the tensors' own
        t.step(x, dout, s)
    t.forward(x, s)
    t.backward(dout)
    leaves = [v.double().requires_grad_() for v in (x, s, w1, b1, w2, gain)]
    r, branch = plain(*leaves)
    r_bf = r + (r.bfloat16().double() - r).detach()  # the stream is kept in bf16
    out = branch + r_bf
    out.backward(dout.double())
    assert torch.equal(t.r, r.bfloat16())
    assert rel(t.out.double() - t.r.double(), branch) < 0.104
    gx, gw1, gb1, gw2, gg = (leaves[i].grad for i in (0, 2, 3, 4, 5))
    assert rel(t.grads[0], gw1) < 0.174 and rel(t.grads[1], gw2) < 0.174
    assert rel(t.grads[2], gg) < 0.174 and rel(t.grads[3], gb1) < 0.174
    assert rel(t.dr.double() - dout.double(), gx - dout.double()) < 0.174
    # the codes the block below starts from
    v = t.drq.view(torch.float8_e5m2).double() * t.scale[B.DR].double()
    assert rel(v, t.dr.double()) < 0.106
    assert F.fp8_get_last_device_error() == (0, 0)


def test_step_in_a_graph():
    """A captured step replays to the same parameters as direct calls."""
    from fp8_quantized_gemm_gb300 import block as B
    w1, b1, w2, gain, rn = make(256, 512)
    x, dout = rn(128, 256).bfloat16(), rn(128, 256, std=1e-2).bfloat16()
    a, b = (B.PreNormMLPTrainer(w1, b1, w2, gain, 128, lr=1e-3) for _ in range(2))
    for t in (a, b):
        t.step(x, dout)
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        b.step(x, dout)
    for _ in range(3):
        a.step(x, dout)
        g.replay()
    for p, q in zip(a.params, b.params):
        assert torch.equal(p, q)
    assert not torch.equal(a.params[0], w1)


@pytest.mark.parametrize("m", [1, 7, 130, 700])
@pytest.mark.parametrize("sfmt", [0, 1])
def test_inference(m, sfmt):
    from fp8_quantized_gemm_gb300 import block as B
    w1, b1, w2, gain, rn = make(512, 1280)
    x, s = rn(m, 512).bfloat16(), rn(m, 512).bfloat16()
    f = B.PreNormMLP(w1, b1, w2, gain, sfmt=sfmt)
    out, r = f(x, s)
    want_r, branch = plain(*[v.double() for v in (x, s, w1, b1, w2, gain)])
    assert torch.equal(r, want_r.bfloat16())
    assert rel(out.double() - r.double(), branch) < 0.104
