"""RMS norm with FP8 output and its gradient against the definitions in 64
bits (plain torch, none of the library's code).

Tolerances.  The kernel forms y in fp32: the sum of K squares is K/threads <= 32
fused steps and a tree of at most 10 more, a relative error of at most 42 x
2^-24 on a sum of positive terms, halved by the square root; the reciprocal
root (2 ulp) and the three products add less than 8 x 2^-24.  REL = 2^-18 covers
it.  A code may then be the rounding of any value that close to y / s: half a
step of the format at y / s, plus REL of it (and the rounding of s itself where
s is formed from the same y).
"""
import math

import pytest
import torch

from gpu_util import lib

pytestmark = pytest.mark.gpu

REL = 2.0 ** -18
F8 = (torch.float8_e4m3fn, torch.float8_e5m2)
TOP = (448.0, 57344.0)
MANT, EMIN = (3, 2), (-6, -14)  # mantissa bits, exponent of the smallest normal
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
EPS = 1e-5


def half_step(v, fmt):
    e = torch.floor(torch.log2(v.abs().clamp_min(2.0 ** EMIN[fmt])))
    return torch.exp2(e - MANT[fmt] - 1)


def check_codes(q, y, s, fmt, rel=REL):
    """q [M, K] uint8 codes of y (f64) under s (f64, broadcast)."""
    v = (y / s).clamp(-TOP[fmt], TOP[fmt])
    got = q.view(F8[fmt]).double()
    bad = (got - v).abs() > half_step(v, fmt) * (1 + 1e-6) + 2 * rel * v.abs()
    assert not bad.any(), (int(bad.sum()), got[bad][:4], v[bad][:4])


def check_ue8m0(bytes_, top, fmt):
    s, e = top / TOP[fmt], bytes_.double() - 127
    zero = top == 0
    assert (e[zero] == 0).all()
    ok = (torch.exp2(e) >= s * (1 - REL)) & (torch.exp2(e - 1) < s * (1 + REL))
    assert (ok | zero).all()


def close(got, want, tol):
    bad = ~((got.double() - want).abs() <= tol)
    assert not bad.any(), (int(bad.sum()), got[bad][:4], want[bad][:4])


def pitched(t, pad):
    """The same matrix with `pad` more elements per row."""
    if not pad:
        return t.contiguous()
    wide = torch.full((t.shape[0], t.shape[1] + pad), 3.0, dtype=t.dtype, device=t.device)
    wide[:, :t.shape[1]] = t
    return wide[:, :t.shape[1]]


def inputs(m, k, dt, wdt, res, seed=0, pad=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    x = rnd(m, k)
    x[:, ::97] *= 30
    x = pitched(x.to(DT[dt]), pad)
    r = pitched((rnd(m, k) * 2).to(DT[dt]), 2 * pad) if res else None
    w = None if wdt is None else (1 + 0.2 * rnd(k)).to(DT[wdt])
    return x, r, w


def definition(x, res, w, eps=EPS):
    r = x.double()
    if res is not None:
        r = (r + res.double()).to(x.dtype).double()
    inv = 1 / torch.sqrt(r.square().mean(1, keepdim=True) + eps)
    return r, inv, r * inv * (1.0 if w is None else w.double())


def tops(y, width):
    m, k = y.shape
    g = (k + width - 1) // width
    return torch.nn.functional.pad(y, (0, g * width - k)).view(m, g, width).abs().amax(2)


SHAPES = [(1, 16), (1, 7168), (3, 128), (2, 16384), (5, 2064), (300, 272), (700, 4096),
          (200, 8208), (160, 16384), (129, 1024), (1000, 480)]


@pytest.mark.parametrize("m,k", SHAPES)
@pytest.mark.parametrize("dt,wdt,res,pad", [("bf16", "f32", True, 0), ("f32", "bf16", True, 8),
                                            ("bf16", "bf16", False, 16), ("f32", None, False, 0)])
@pytest.mark.parametrize("mode", ["tensor", "f32", "ue8m0", "mx"])
def test_forward(m, k, dt, wdt, res, pad, mode):
    if mode == "mx" and k % 128:
        pytest.skip("MX words cover 128-wide slices")
    F = lib()
    fmt = m % 2
    x, rs, w = inputs(m, k, dt, wdt, res, seed=m + k, pad=pad)
    r, inv, y = definition(x, rs, w)
    new = lambda *s, t=torch.float32: torch.empty(*s, dtype=t, device="cuda")  # noqa: E731
    q, inv_out, y_out = new(m, k, t=torch.uint8), new(m), new(m, k, t=torch.bfloat16)
    s_out = pitched(new(m, k, t=x.dtype), pad)
    kw = dict(residual=rs, sum_out=s_out, y_out=y_out, inv_rms=inv_out)
    if mode == "tensor":
        scale, amax = torch.full((1,), 9.0 / TOP[fmt], device="cuda"), new(1)
        F.fp8_rmsnorm_quantize(x, w, EPS, fmt, q, scale=scale, amax_out=amax, **kw)
        check_codes(q, y, scale.double(), fmt)
        close(amax, y.abs().max().reshape(1), REL * y.abs().max())
    elif mode == "mx":
        words = F.mx_local_words(m, k)
        words.fill_(-1)
        F.fp8_rmsnorm_quantize(x, w, EPS, fmt, q, local=words, **kw)
        from gpu_util import mx_unpack
        b = torch.from_numpy(mx_unpack(words.cpu().numpy(), m, k)).cuda()
        check_ue8m0(b, tops(y, 32), fmt)
        check_codes(q, y, torch.exp2(b.double() - 127).repeat_interleave(32, 1), fmt)
        pad_rows = torch.arange(m, (m + 127) // 128 * 128)
        at = (pad_rows & ~127) + 4 * (pad_rows % 32) + (pad_rows % 128) // 32
        assert (words.cpu()[:, at] == 0x7F7F7F7F).all()
    else:
        g = (k + 127) // 128
        top = tops(y, 128)
        if mode == "f32":
            sc = new(g, m)
            F.fp8_rmsnorm_quantize(x, w, EPS, fmt, q, scales=sc, **kw)
            s = sc.t().double()
            close(s, top / TOP[fmt], REL * top / TOP[fmt])
        else:
            sc = new(g, m, t=torch.uint8)
            F.fp8_rmsnorm_quantize(x, w, EPS, fmt, q, scales=sc, sfmt=F.SCALE_UE8M0, **kw)
            check_ue8m0(sc.t(), top, fmt)
            s = torch.exp2(sc.t().double() - 127)
        check_codes(q, y, s.repeat_interleave(128, 1)[:, :k], fmt)
    assert torch.equal(s_out.double(), r)
    close(inv_out, inv[:, 0], REL * inv[:, 0])
    close(y_out, y, (REL + 2.0 ** -8) * y.abs() + 1e-38)


def test_forward_in_place_and_deterministic():
    """The sum may overwrite the residual; the same call gives the same bits."""
    F = lib()
    m, k = 333, 2048
    x, rs, w = inputs(m, k, "bf16", "f32", True)
    outs = []
    for inplace in (False, True):
        stream = rs.clone()
        s_out = stream if inplace else torch.empty_like(rs)
        q, sc = torch.empty((m, k), dtype=torch.uint8, device="cuda"), torch.empty((16, m), device="cuda")
        F.fp8_rmsnorm_quantize(x, w, EPS, F.E4M3, q, residual=stream, sum_out=s_out, scales=sc)
        outs.append((q, sc, s_out))
    for a, b in zip(*outs):
        assert torch.equal(a, b)


@pytest.mark.parametrize("mode", ["tensor", "f32", "ue8m0", "mx"])
def test_special_rows(mode):
    """Zero rows give zero codes and unit scales; a NaN or infinity reaches its
    own row only."""
    F = lib()
    m, k = 6, 256
    x = torch.randn(m, k, device="cuda")
    x[1] = 0
    x[2, 77] = float("nan")
    x[4, 5] = float("inf")
    q = torch.empty((m, k), dtype=torch.uint8, device="cuda")
    one = torch.full((1,), 0.02, device="cuda")
    kw = {"tensor": dict(scale=one), "f32": dict(scales=torch.empty((2, m), device="cuda")),
          "ue8m0": dict(scales=torch.empty((2, m), dtype=torch.uint8, device="cuda"),
                        sfmt=F.SCALE_UE8M0), "mx": dict(local=F.mx_local_words(m, k))}[mode]
    F.fp8_rmsnorm_quantize(x, None, EPS, F.E4M3, q, **kw)
    v = q.view(F8[0]).float()
    assert (v[1] == 0).all()
    if mode == "f32":
        assert (kw["scales"][:, 1] == 1).all()
    if mode == "ue8m0":
        assert (kw["scales"][:, 1] == 127).all()
    assert torch.isnan(v[2]).all() and torch.isnan(v[4, 5])
    for row in (0, 3, 5):
        assert torch.isfinite(v[row]).all() and (v[row] != 0).any()


def test_no_rows():
    F = lib()
    k = 64
    x, q = torch.empty((0, k), device="cuda"), torch.empty((0, k), dtype=torch.uint8, device="cuda")
    amax, scale = torch.full((1,), 5.0, device="cuda"), torch.ones(1, device="cuda")
    F.fp8_rmsnorm_quantize(x, None, EPS, F.E4M3, q, scale=scale, amax_out=amax)
    assert amax.item() == 0
    dw = torch.ones(k, device="cuda")
    F.fp8_rmsnorm_backward(x, x, torch.empty(0, device="cuda"), None, torch.empty_like(x), dw=dw)
    assert (dw == 0).all()


@pytest.mark.parametrize("m,k", SHAPES)
@pytest.mark.parametrize("dt,dydt,wdt,dres,codes,pad", [
    ("bf16", "bf16", "f32", True, True, 0), ("f32", "f32", "bf16", True, False, 8),
    ("bf16", "f32", "bf16", False, True, 16), ("f32", "bf16", None, False, False, 0)])
def test_backward(m, k, dt, dydt, wdt, dres, codes, pad):
    F = lib()
    r, e, w = inputs(m, k, dt, wdt, dres, seed=m * 7 + k, pad=pad)
    gen = torch.Generator(device="cuda").manual_seed(5)
    dy = pitched(torch.randn(m, k, generator=gen, device="cuda").to(DT[dydt]), pad)
    inv = torch.rsqrt(r.double().square().mean(1) + EPS).float()
    dx, dw = pitched(torch.empty(m, k, dtype=r.dtype, device="cuda"), pad), torch.ones(k, device="cuda")
    fmt, kw = F.E5M2, {}
    if codes:
        kw = dict(q=torch.empty((m, k), dtype=torch.uint8, device="cuda"), fmt=fmt,
                  scale=torch.full((1,), 30.0 / TOP[fmt], device="cuda"),
                  amax_out=torch.empty(1, device="cuda"))
    F.fp8_rmsnorm_backward(dy, r, inv, w, dx, d_residual=e, dw=dw, accumulate_dw=True, **kw)
    D = lambda t: t.double()  # noqa: E731
    i, g = D(inv)[:, None], D(dy) * (1.0 if w is None else D(w))
    xh = D(r) * i
    want = i * (g - xh * (g * xh).mean(1, keepdim=True)) + (0 if e is None else D(e))
    # fp32 chains of at most 42 steps on each term, plus the output's rounding
    size = i * (g.abs() + xh.abs() * (g * xh).abs().mean(1, keepdim=True)) + \
        (0 if e is None else D(e).abs())
    tol = 42 * 2.0 ** -24 * size + 1e-38
    close(dx, want, tol + (2.0 ** -8 if dt == "bf16" else 2.0 ** -23) * want.abs())
    # at most m sequential additions and two short trees
    terms = (D(dy) * xh).abs().sum(0)
    close(dw, (D(dy) * xh).sum(0) + 1, (m + 32) * 2.0 ** -24 * (terms + 1))
    if codes:
        s = D(kw["scale"])
        v = (want / s).clamp(-TOP[fmt], TOP[fmt])
        got = kw["q"].view(F8[fmt]).double()
        assert ((got - v).abs() <= half_step(v.abs() + tol / s, fmt) * (1 + 1e-6) + 2 * tol / s).all()
        close(kw["amax_out"], want.abs().max().reshape(1), tol.max())


def test_backward_against_differences():
    """dx and dw against central differences of sum(dy y) in 64 bits."""
    F = lib()
    m, k, h = 3, 48, 1e-6
    r, _, w = inputs(m, k, "f32", "f32", False, seed=9)
    dy = torch.randn(m, k, device="cuda")
    inv = torch.rsqrt(r.square().mean(1) + EPS)
    dx, dw = torch.empty_like(r), torch.empty(k, device="cuda")
    F.fp8_rmsnorm_backward(dy, r, inv, w, dx, dw=dw)

    def loss(rr, ww):
        return (dy.double() * rr * ww / torch.sqrt(rr.square().mean(-1, keepdim=True) + EPS)).sum((-1, -2))

    rd, wd = r.double(), w.double()
    step = h * torch.eye(m * k, device="cuda", dtype=torch.float64).view(m * k, m, k)
    num = ((loss(rd + step, wd) - loss(rd - step, wd)) / (2 * h)).view(m, k)
    ws = h * torch.eye(k, device="cuda", dtype=torch.float64).view(k, 1, k)
    numw = (loss(rd, wd + ws) - loss(rd, wd - ws)) / (2 * h)
    # differences: truncation ~h^2, cancellation ~1e-16 |loss| / h ~ 1e-8; fp32 terms 1e-5
    close(dx, num, 1e-5 * (1 + num.abs()))
    close(dw, numw, 1e-5 * (1 + numw.abs()))


def test_backward_in_place_repeatable_other_stream():
    """dx over d_residual, on a side stream with its own workspace: the bits of
    the plain call (no atomics in dw)."""
    F = lib()
    m, k = 1500, 2048
    r, e, w = inputs(m, k, "bf16", "f32", True, seed=3)
    e = e.contiguous()
    dy = torch.randn(m, k, device="cuda").bfloat16()
    inv = torch.rsqrt(r.float().square().mean(1) + EPS)
    dx, dw = torch.empty_like(r), torch.empty(k, device="cuda")
    F.fp8_rmsnorm_backward(dy, r, inv, w, dx, d_residual=e, dw=dw)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    dw2 = torch.empty_like(dw)
    ws = torch.empty(F.fp8_rmsnorm_backward_workspace(m, k), dtype=torch.uint8, device="cuda")
    with pytest.raises(ValueError):
        F.fp8_rmsnorm_backward(dy, r, inv, w, e, d_residual=e, dw=dw2, stream=side)
    F.fp8_rmsnorm_backward(dy, r, inv, w, e, d_residual=e, dw=dw2, workspace=ws, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(e, dx) and torch.equal(dw, dw2)


def test_long_matrix_offsets():
    """Rows whose element offsets pass 2^31."""
    F = lib()
    k, m = 16384, 131073 + 8
    x = torch.zeros((m, k), dtype=torch.bfloat16, device="cuda")
    x[-9:] = torch.randn(9, k, device="cuda").bfloat16()
    q = torch.empty((m, k), dtype=torch.uint8, device="cuda")
    sc = torch.empty((k // 128, m), device="cuda")
    F.fp8_rmsnorm_quantize(x, None, EPS, F.E4M3, q, scales=sc)
    _, _, y = definition(x[-9:], None, None)
    check_codes(q[-9:], y, sc[:, -9:].t().double().repeat_interleave(128, 1), 0)
    assert (q[:-9] == 0).all() and (sc[:, :-9] == 1).all()


def test_graph_capture():
    F = lib()
    m, k = 64, 1024
    x, rs, w = inputs(m, k, "bf16", "f32", True)
    q, amax = torch.empty((m, k), dtype=torch.uint8, device="cuda"), torch.empty(1, device="cuda")
    s_out, scale = torch.empty_like(rs), torch.full((1,), 0.03, device="cuda")
    call = lambda: F.fp8_rmsnorm_quantize(x, w, EPS, F.E4M3, q, residual=rs, sum_out=s_out,  # noqa: E731
                                          scale=scale, amax_out=amax)
    call()
    ref = q.clone()
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        call()
    q.zero_()
    amax.zero_()
    g.replay()
    assert torch.equal(q, ref) and math.isfinite(amax.item()) and amax.item() > 0
