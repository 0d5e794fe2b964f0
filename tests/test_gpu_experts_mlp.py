"""The mixture-of-experts layer as a run of the calls: outputs and gradients
against the same layer in 64 bits on the values of the quantized weights.

Tolerances (2-norm of the difference over the norm of the result).  A code is
off by at most 2^-4 of its value, and independent errors add up to no more than
that much of a product's norm.  On the way forward x, a and (through a = act(h)
u, whose relative error is about that of its two arguments) h and u carry it:
3 x 2^-4.  On the way back w dout, the checkpoints of h and u and dh | du do:
4 x 2^-4.  (A row of another token, expert or weight is off by 1.4.)
"""
import pytest
import torch

from gpu_util import lib

pytestmark = pytest.mark.gpu

BF = torch.bfloat16
F8 = torch.float8_e4m3fn


def randn(shape, seed, std):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(shape, generator=g, device="cuda") * std


def values(pair, sfmt):
    """64-bit values of block-scaled weights."""
    q, s = pair
    s = torch.exp2(s.double() - 127) if sfmt else s.double()
    s = s.repeat_interleave(128, 1).repeat_interleave(128, 2)
    return q.view(F8).double() * s


def act(z, name):
    if name == "relu2":
        return z.clamp_min(0) ** 2
    return z * torch.sigmoid(z)


def layer(x, w, ids, w13, w2, name, residual):
    """out of the layer in 64 bits."""
    e, n = w13.shape[0], w13.shape[1] // 2
    out = torch.zeros_like(x) if residual is None else residual
    for i in range(e):
        t, s = torch.nonzero(ids == i, as_tuple=True)
        if t.numel() == 0:
            continue
        hu = x[t] @ w13[i].t()
        y = (act(hu[:, :n], name) * hu[:, n:]) @ w2[i].t()
        out = out.index_add(0, t, y * w[t, s][:, None])
    return out


def far(got, want):
    return float((got.double() - want).norm() / want.norm().clamp_min(1e-30))


CASES = [  # t, s, e, d, ffn, drop, sfmt, keep_sfmt, act, residual
    (1, 2, 4, 256, 128, 0.0, 0, 0, "silu", False), (37, 3, 5, 256, 384, 0.3, 0, 1, "silu", True),
    (200, 2, 8, 512, 256, 0.0, 1, 0, "relu2", True), (700, 4, 16, 1024, 512, 0.2, 1, 1, "silu", False),
    (700, 4, 16, 1024, 512, 0.0, 0, 0, "silu", True)]


@pytest.mark.parametrize("t,s,e,d,ffn,drop,sfmt,keep_sfmt,name,res", CASES)
def test_layer(t, s, e, d, ffn, drop, sfmt, keep_sfmt, name, res):
    F = lib()
    from fp8_quantized_gemm_gb300.experts import ExpertsMLP
    w13 = randn((e, 2 * ffn, d), 1, d ** -0.5).to(BF)
    w2 = randn((e, d, ffn), 2, ffn ** -0.5).to(BF)
    mlp = ExpertsMLP(w13, w2, act=F.ACT_RELU2 if name == "relu2" else F.ACT_SILU, sfmt=sfmt,
                     backward=True, keep_sfmt=keep_sfmt)
    x = randn((t, d), 3, 1.0).to(BF)
    w = torch.softmax(randn((t, s), 4, 1.0), 1)
    ids = torch.randint(0, e, (t, s), device="cuda", generator=torch.Generator("cuda").manual_seed(5))
    if drop:
        u = torch.rand((t, s), device="cuda", generator=torch.Generator("cuda").manual_seed(6))
        ids = torch.where(u < drop, e + 3, ids)
        ids[0] = -1  # a token that no expert takes
    r = randn((t, d), 7, 1.0).to(BF) if res else None
    out = mlp(x, ids, w, residual=r, keep=True)
    xd, wd = x.double().requires_grad_(True), w.double().requires_grad_(True)
    want = layer(xd, wd, ids, values(mlp.w13, sfmt), values(mlp.w2, sfmt), name,
                 None if r is None else r.double())
    part = want.detach() - (0 if r is None else r.double())
    got = out.double() - (0 if r is None else r.double())
    # (the output's own rounding is of the sum with the residual)
    slack = 2.0 ** -8 * float(want.norm() / part.norm())
    assert far(got, part) <= 3 * 2.0 ** -4 + slack
    dout = randn((t, d), 8, 1e-2).to(BF)
    gx, gw = torch.autograd.grad(want, (xd, wd), dout.double(), retain_graph=True)
    dx, dw = mlp.backward(dout)
    # the transposed weights' codes stand for the same values
    assert torch.equal(values(mlp.w13t, sfmt), values(mlp.w13, sfmt).transpose(1, 2))
    assert far(dx, gx) <= 4 * 2.0 ** -4 + 2.0 ** -8 and far(dw, gw) <= 3 * 2.0 ** -4 + 2.0 ** -8
    dropped = (ids < 0) | (ids >= e)
    assert (dw[dropped] == 0).all()
    if drop:
        assert (dx[0] == 0).all() and torch.equal(out[0], r[0] if res else torch.zeros_like(out[0]))
    # int32 ids, and codes that exist already: the same bits
    st = torch.uint8 if sfmt else torch.float32
    xq, xs = torch.empty((t, d), dtype=torch.uint8, device="cuda"), torch.empty((d // 128, t), dtype=st, device="cuda")
    F.fp8_quantize_token_group(x, F.E4M3, sfmt, xq, xs)
    assert torch.equal(mlp(xq, ids.int(), w, x_scales=xs, residual=r), out)


def test_no_tokens_and_refusals():
    F = lib()
    from fp8_quantized_gemm_gb300.experts import ExpertsMLP
    w13, w2 = randn((2, 256, 128), 1, 0.1).to(BF), randn((2, 128, 128), 2, 0.1).to(BF)
    mlp = ExpertsMLP(w13, w2)
    x = randn((3, 128), 3, 1.0).to(BF)
    empty = torch.empty((0, 2), device="cuda")
    assert mlp(x[:0], empty.long(), empty).shape == (0, 128)
    grad = ExpertsMLP(w13, w2, backward=True)
    grad(x[:0], empty.long(), empty, keep=True)
    dx, dw = grad.backward(x[:0])
    assert dx.shape == (0, 128) and dw.shape == (0, 2)
    ids = torch.full((3, 2), -1, dtype=torch.int64, device="cuda")
    assert (mlp(x, ids, torch.ones((3, 2), device="cuda")) == 0).all()  # no expert takes any
    with pytest.raises(ValueError):
        mlp.backward(x)
    with pytest.raises(ValueError):
        ExpertsMLP(w13[:, :200], w2)
    assert F.fp8_get_last_device_error() == (0, 0)


@pytest.mark.parametrize("sfmt", [0, 1])
def test_captured_layer(sfmt):
    """Forward and backward captured once, replayed on other tokens and choices."""
    lib()
    from fp8_quantized_gemm_gb300.experts import ExpertsMLP
    t, s, e, d, ffn = 300, 2, 8, 256, 256
    mlp = ExpertsMLP(randn((e, 2 * ffn, d), 1, d ** -0.5).to(BF),
                     randn((e, d, ffn), 2, ffn ** -0.5).to(BF), sfmt=sfmt, backward=True)
    sets = []
    for i in range(2):
        gen = torch.Generator("cuda").manual_seed(40 + i)
        sets.append((randn((t, d), 10 + i, 1.0).to(BF), torch.randint(-1, e, (t, s), generator=gen, device="cuda"),
                     torch.softmax(randn((t, s), 20 + i, 1.0), 1), randn((t, d), 30 + i, 1e-2).to(BF)))
    want = []
    for x, ids, w, dout in sets:
        out = mlp(x, ids, w, keep=True)
        want.append((out,) + mlp.backward(dout))
    live = [v.clone() for v in sets[0]]
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = mlp(live[0], live[1], live[2], keep=True)
        dx, dw = mlp.backward(live[3])
    for i in (1, 0):
        for v, src in zip(live, sets[i]):
            v.copy_(src)
        g.replay()
        torch.cuda.synchronize()
        for a, b in zip((out, dx, dw), want[i]):
            assert torch.equal(a, b)
