"""GEMM with bias, activation, residual and FP8 output in its epilogue, and the
activation-gradient GEMM, against the definitions in 64 bits (plain torch, none
of the library's code).

Tolerances.  z: an fp32 accumulation of K products in any order, each step
within 2^-23 of the running magnitude: (K + 8) 2^-23 sum |a||b| (scaled), plus
the bias' rounding.  y: that times the activation's largest slope nearby
(1.13 for the smooth ones, 2 |z| + ... for relu2), the fp32 arithmetic of the
activation within 2^-18 of |z| + |y|, then the rounding of the stored type
(bf16: 2^-8, fp32: 2^-23 of the value) or half a step of the code.
"""
import math

import pytest
import torch

from gpu_util import lib
from test_gpu_rmsnorm import F8, TOP, close, half_step, pitched

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
ACTS = ["none", "relu", "relu2", "silu", "gelu_tanh", "gelu"]


def act64(z, name):
    phi = 0.5 * torch.erfc(-z / math.sqrt(2))
    if name == "relu":
        return z.clamp_min(0), (z > 0).double()
    if name == "relu2":
        return z.clamp_min(0) ** 2, 2 * z.clamp_min(0)
    if name == "silu":
        s = torch.sigmoid(z)
        return z * s, s * (1 + z * (1 - s))
    if name == "gelu_tanh":
        a = math.sqrt(2 / math.pi)
        t = torch.tanh(a * (z + 0.044715 * z ** 3))
        return 0.5 * z * (1 + t), 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * a * (1 + 3 * 0.044715 * z * z)
    if name == "gelu":
        return z * phi, phi + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    return z, torch.ones_like(z)


def randn(*shape, seed=0, std=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(*shape, generator=g, device="cuda") * std


def codes(t, fmt):
    s = (t.abs().max() / TOP[fmt]).reshape(1)
    return (t / s).clamp(-TOP[fmt], TOP[fmt]).to(F8[fmt]).view(torch.uint8), s


def value(q, fmt):
    return q.view(F8[fmt]).double()


def check_epilogue(c, y, tz, z, name, out, pre, q, qs, amax, fmt):
    slope = torch.where(z > -50, 2 * (z.abs() + tz), z * 0) if name == "relu2" else 1.13
    ty = slope * tz + 2.0 ** -18 * (z.abs() + y.abs()) + 1e-30
    if pre is not None:
        close(pre, z, tz + 2.0 ** -8 * (z.abs() + tz))
    if out is not None:
        close(out, y, ty + (2.0 ** -8 if out.dtype == torch.bfloat16 else 2.0 ** -23) * (y.abs() + ty))
    if q is not None:
        s = qs.double()
        v = (y / s).clamp(-TOP[fmt], TOP[fmt])
        assert ((value(q, fmt) - v).abs() <= half_step(v.abs() + ty / s, fmt) * (1 + 1e-6) + 2 * ty / s).all()
        close(amax, y.abs().max().reshape(1), ty.max())


# one tile and less, ragged tiles, split K in a cluster, CTA pairs
TENSOR = [(1, 1, 16), (3, 8, 48), (37, 65, 144), (130, 257, 272), (33, 520, 2064), (1, 2048, 4096),
          (700, 300, 1040), (1029, 1283, 272), (2048, 2560, 160)]
VARIANTS = [  # bias, residual, its pitch, out, pre, codes
    (True, "bf16", 0, "bf16", False, False), (False, "f32", 3, "f32", True, False),
    (True, None, 0, None, True, True), (True, "bf16", 1, "bf16", True, True),
    (False, None, 0, "f32", False, False)]


@pytest.mark.parametrize("m,n,k", TENSOR)
@pytest.mark.parametrize("v", range(len(VARIANTS)))
@pytest.mark.parametrize("name", ACTS)
def test_tensor(m, n, k, v, name):
    F = lib()
    bias, res, pad, out, pre, cod = VARIANTS[v]
    fa, fb, fq = v % 2, (v // 2) % 2, (v + 1) % 2
    a, sa = codes(randn(m, k, seed=m + v), fa)
    b, sb = codes(randn(n, k, seed=n + 1, std=1.5 / math.sqrt(k)), fb)
    bs = randn(n, seed=3, std=0.5) if bias else None
    r = pitched(randn(m, n, seed=4).to(DT[res]), pad) if res else None
    c = pitched(torch.empty(m, n, dtype=DT[out], device="cuda"), pad) if out else None
    p = pitched(torch.empty(m, n, dtype=torch.bfloat16, device="cuda"), pad) if pre else None
    kw = {}
    if cod:
        kw = dict(q=torch.empty((m, n), dtype=torch.uint8, device="cuda"), q_fmt=fq,
                  q_scale=torch.full((1,), 6.0 / TOP[fq], device="cuda"),
                  q_amax=torch.full((1,), 1e30, device="cuda"))
    F.fp8_gemm_tensor_epilogue(a, fa, b, fb, sa, sb, c, bias=bs, act=ACTS.index(name), residual=r,
                               pre_out=p, **kw)
    A, B, al = value(a, fa), value(b, fb), sa.double() * sb.double()
    z = A @ B.t() * al + (0 if bs is None else bs.double())
    tz = (k + 8) * 2.0 ** -23 * (A.abs() @ B.abs().t() * al) + 2.0 ** -23 * z.abs()
    y = act64(z, name)[0] + (0 if r is None else r.double())
    tr = tz + (0 if r is None else 2.0 ** -23 * r.double().abs())
    check_epilogue(None, y, tr, z, name, c, p, kw.get("q"), kw.get("q_scale"), kw.get("q_amax"), fq)
    assert F.fp8_get_last_device_error() == (0, 0)


@pytest.mark.parametrize("m,n,k", [(48, 64, 80), (1040, 1280, 272), (32, 528, 2064)])
def test_tensor_mn_major(m, n, k):
    """Operands read transposed, residual added in place."""
    F = lib()
    a, sa = codes(randn(k, m, seed=1), 1)
    b, sb = codes(randn(k, n, seed=2, std=1 / math.sqrt(k)), 0)
    c = randn(m, n, seed=3).bfloat16()
    r0 = c.double()
    F.fp8_gemm_tensor_epilogue(a, 1, b, 0, sa, sb, c, act=F.ACT_SILU, residual=c,
                               a_layout=F.MN_MAJOR, b_layout=F.MN_MAJOR)
    A, B, al = value(a, 1).t(), value(b, 0).t(), sa.double() * sb.double()
    z = A @ B.t() * al
    tz = (k + 8) * 2.0 ** -23 * (A.abs() @ B.abs().t() * al) + 2.0 ** -23 * r0.abs()
    check_epilogue(None, act64(z, "silu")[0] + r0, tz, z, "silu", c, None, None, None, None, 0)


def group_operands(m, n, k, sfmt):
    g, nb = k // 128, (n + 127) // 128
    x = randn(m, k, seed=m)
    x[:, ::61] *= 20
    w = torch.zeros(nb * 128, k, device="cuda")
    w[:n] = randn(n, k, seed=n, std=1.5 / math.sqrt(k))

    def scales(top):
        s = torch.where(top > 0, top / 448, torch.ones_like(top))
        if sfmt == 0:
            return s, s
        e = torch.ceil(torch.log2(s.double()))
        return torch.exp2(e).float(), (e + 127).to(torch.uint8)

    sx, kx = scales(x.view(m, g, 128).abs().amax(2))
    sw, kw = scales(w.view(nb, 128, g, 128).abs().amax((1, 3)))
    q = lambda t: t.clamp(-448, 448).to(F8[0])  # noqa: E731
    a = q(x.view(m, g, 128) / sx[..., None])
    b = q(w.view(nb, 128, g, 128) / sw[:, None, :, None])
    A = (a.double() * sx.double()[..., None]).view(m, k)
    B = (b.double() * sw.double()[:, None, :, None]).view(nb * 128, k)[:n]
    u8 = torch.uint8
    return (a.view(m, k).view(u8), kx.t().contiguous(),
            b.view(nb * 128, k)[:n].contiguous().view(u8), kw.contiguous(), A, B)


@pytest.mark.parametrize("m,n,k", [(1, 1, 128), (1, 2048, 7168), (17, 65, 384), (33, 1283, 1024),
                                   (100, 300, 2048), (200, 384, 1024), (300, 1100, 512),
                                   (2051, 1283, 256), (1500, 2600, 256),
                                   (2200, 2600, 384)])
@pytest.mark.parametrize("sfmt", [0, 1])
@pytest.mark.parametrize("name,bias,res,pad,pre", [
    ("none", True, "bf16", 0, False), ("silu", False, "f32", 3, True),
    ("gelu", True, None, 1, True), ("relu2", True, "bf16", 8, False),
    ("gelu_tanh", False, None, 0, False), ("relu", True, "f32", 0, True)])
def test_group(m, n, k, sfmt, name, bias, res, pad, pre):
    F = lib()
    a, sa, b, sb, A, B = group_operands(m, n, k, sfmt)
    bs = randn(n, seed=3, std=0.5) if bias else None
    r = pitched(randn(m, n, seed=4).to(DT[res]), pad) if res else None
    c = pitched(torch.empty(m, n, dtype=torch.bfloat16, device="cuda"), pad)
    p = pitched(torch.empty(m, n, dtype=torch.bfloat16, device="cuda"), pad) if pre else None
    F.fp8_gemm_group_epilogue(a, sa, b, sb, sfmt, c, bias=bs, act=ACTS.index(name), residual=r,
                              pre_out=p)
    z = A @ B.t() + (0 if bs is None else bs.double())
    tz = (k + 8) * 2.0 ** -23 * (A.abs() @ B.abs().t()) + 2.0 ** -23 * z.abs()
    y = act64(z, name)[0] + (0 if r is None else r.double())
    tr = tz + (0 if r is None else 2.0 ** -23 * r.double().abs())
    check_epilogue(None, y, tr, z, name, c, p, None, None, None, 0)
    assert F.fp8_get_last_device_error() == (0, 0)


@pytest.mark.parametrize("m,n,k,mn", [(1, 16, 16, True), (5, 33, 48, False), (333, 1040, 528, True),
                                      (700, 144, 272, True), (1029, 1283, 272, False),
                                      (64, 256, 2064, True)])
@pytest.mark.parametrize("name", ACTS)
@pytest.mark.parametrize("out,pad", [("bf16", 0), ("f32", 3), (None, 0)])
def test_act_backward(m, n, k, mn, name, out, pad):
    F = lib()
    a, sa = codes(randn(m, k, seed=m, std=1e-3), 1)
    b, sb = codes(randn(k, n, seed=n, std=1 / math.sqrt(n)), 0)
    B = value(b, 0)
    if not mn:
        b = b.t().contiguous()
    pre = pitched(randn(m, n, seed=5, std=1.5).bfloat16(), pad)
    c = pitched(torch.empty(m, n, dtype=DT[out], device="cuda"), pad) if out else None
    db = torch.full((n,), 0.25, device="cuda")
    acc = out == "f32"
    kw = {}
    if out != "f32":
        kw = dict(q=torch.empty((m, n), dtype=torch.uint8, device="cuda"), q_fmt=F.E5M2,
                  q_scale=torch.full((1,), 5e-3 / TOP[1], device="cuda"),
                  q_amax=torch.empty(1, device="cuda"))
    F.fp8_gemm_tensor_act_backward(a, 1, b, 0, sa, sb, pre, ACTS.index(name), out=c, dbias=db,
                                   accumulate_dbias=acc, b_layout=F.MN_MAJOR if mn else F.K_MAJOR,
                                   **kw)
    A, al = value(a, 1), sa.double() * sb.double()
    g, slope = A @ B * al, act64(pre.double(), name)[1]
    tg = (k + 8) * 2.0 ** -23 * (A.abs() @ B.abs() * al)
    want = g * slope
    tol = tg * slope.abs() + 2.0 ** -18 * g.abs() * (1 + slope.abs()) + 1e-30
    if c is not None:
        close(c, want, tol + (2.0 ** -8 if out == "bf16" else 2.0 ** -23) * (want.abs() + tol))
    if kw:
        s = kw["q_scale"].double()
        v = (want / s).clamp(-TOP[1], TOP[1])
        assert ((value(kw["q"], 1) - v).abs() <=
                half_step(v.abs() + tol / s, 1) * (1 + 1e-6) + 2 * tol / s).all()
        close(kw["q_amax"], want.abs().max().reshape(1), tol.max())
    # ceil(m / 32) partial sums of 32 terms
    close(db, want.sum(0) + (0.25 if acc else 0),
          tol.sum(0) + (m + 64) * 2.0 ** -24 * (want.abs().sum(0) + 0.25))


@pytest.mark.parametrize("name", ACTS[1:])
def test_slope_against_differences(name):
    """act' of the gradient call against central differences of the activation
    that the forward call applies (both read through identity products)."""
    F = lib()
    m, n = 64, 64
    z = torch.linspace(-8, 8, m * n, device="cuda").view(m, n).bfloat16()
    z[z.abs() < 0.05] = 0.5  # away from relu's corner
    eye, one = codes(torch.eye(m, device="cuda"), 0)
    zero = torch.zeros((n, m), dtype=torch.uint8, device="cuda")
    h = 2.0 ** -6

    def forward(bias_shift):
        # act(z + shift): z enters as the residual-free pre-activation through
        # one row at a time of the bias
        out = torch.empty((m, n), device="cuda")
        for i in range(m):
            F.fp8_gemm_tensor_epilogue(eye[:1], 0, zero, 0, one, one, out[i:i + 1],
                                       bias=(z[i].float() + bias_shift).contiguous(),
                                       act=ACTS.index(name))
        return out.double()

    num = (forward(h) - forward(-h)) / (2 * h)
    ones, s1 = codes(torch.ones((m, 16), device="cuda") / 16, 0)
    onesb, s2 = codes(torch.ones((n, 16), device="cuda"), 0)
    got = torch.empty((m, n), device="cuda")
    F.fp8_gemm_tensor_act_backward(ones, 0, onesb, 0, s1, s2, z, ACTS.index(name), out=got)
    # truncation: h^2 / 6 |act'''| (< 2) = 8e-5; cancellation: 2^-20 |act| / h < 5e-4
    close(got, num, 1e-3 * (1 + num.abs()))


@pytest.mark.parametrize("name", ACTS[1:])
def test_extreme_arguments(name):
    """Large, tiny and NaN pre-activations: the limits, no NaN of their own."""
    F = lib()
    z = torch.tensor([3e38, -3e38, 1e20, -1e20, 1e4, -1e4, 90, -90, 20, -20, 1e-30, -1e-30, 0.0, -0.0,
                      float("nan"), 1.0], device="cuda")
    a, s = torch.zeros((1, 16), dtype=torch.uint8, device="cuda"), torch.ones(1, device="cuda")
    b = torch.zeros((16, 16), dtype=torch.uint8, device="cuda")
    out = torch.empty((1, 16), device="cuda")
    F.fp8_gemm_tensor_epilogue(a, 0, b, 0, s, s, out, bias=z, act=ACTS.index(name))
    want = act64(z.double().clamp(-1e4, 1e4), name)[0]
    big = z.abs() > 1e4
    fin = ~torch.isnan(z) & ~(big & (name == "relu2"))
    want = torch.where(big, z.double().clamp_min(0), want)
    close(out[0][fin], want[fin], 2.0 ** -17 * want[fin].abs() + 1e-30 * 0 + 1e-7)
    assert torch.isnan(out[0, 14])
    g = torch.empty((1, 16), device="cuda")
    ones, s1 = codes(torch.ones((1, 16), device="cuda"), 0)
    onesb, s2 = codes(torch.ones((16, 16), device="cuda") / 16, 0)
    F.fp8_gemm_tensor_act_backward(ones, 0, onesb, 0, s1, s2, z.bfloat16()[None], ACTS.index(name), out=g)
    zb = z.bfloat16().double()
    slope = act64(zb.clamp(-1e4, 1e4), name)[1]
    if name == "relu2":
        slope = (2 * zb.clamp_min(0)).float().double()  # 2 x 3e38 is past fp32: infinite
    ok = torch.isfinite(slope) & ~torch.isnan(zb)
    assert torch.equal(g[0].double()[torch.isinf(slope)], slope[torch.isinf(slope)])
    close(g[0][ok], slope[ok], 2.0 ** -17 * slope[ok].abs() + 1e-6)
    assert torch.isnan(g[0, 14])


def test_other_stream_and_graph():
    F = lib()
    m, n, k = 512, 2560, 256
    a, sa = codes(randn(m, k), 0)
    b, sb = codes(randn(n, k, seed=1), 0)
    pre = randn(m, n, seed=2).bfloat16()
    side = torch.cuda.Stream()
    ref, got, db, db2 = (torch.empty((m, n), device="cuda", dtype=torch.bfloat16) for _ in range(2)), None, \
        torch.empty(n, device="cuda"), torch.empty(n, device="cuda")
    ref, got = ref
    F.fp8_gemm_tensor_act_backward(a, 0, b, 0, sa, sb, pre, F.ACT_GELU, out=ref, dbias=db)
    ws = torch.empty(F.fp8_act_backward_workspace(m, n), dtype=torch.uint8, device="cuda")
    side.wait_stream(torch.cuda.current_stream())
    F.fp8_gemm_tensor_act_backward(a, 0, b, 0, sa, sb, pre, F.ACT_GELU, out=got, dbias=db2,
                                   workspace=ws, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(ref, got) and torch.equal(db, db2)
    got.zero_()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        F.fp8_gemm_tensor_act_backward(a, 0, b, 0, sa, sb, pre, F.ACT_GELU, out=got, dbias=db2,
                                       workspace=ws)
    db2.zero_()
    g.replay()
    assert torch.equal(ref, got) and torch.equal(db, db2)


def run_plain_epilogue(m, n, k, grad):
    """One call with bf16 output; returns (output, exact, tolerance)."""
    F = lib()
    a, sa = codes(randn(m, k, seed=1), 0)
    b, sb = codes(randn(n, k, seed=2, std=1 / math.sqrt(k)), 0)
    pre = randn(m, n, seed=3).bfloat16()
    out = torch.empty((m, n), dtype=torch.bfloat16, device="cuda")
    if grad:
        F.fp8_gemm_tensor_act_backward(a, 0, b, 0, sa, sb, pre, F.ACT_RELU, out=out)
    else:
        F.fp8_gemm_tensor_epilogue(a, 0, b, 0, sa, sb, out, act=F.ACT_RELU, residual=pre)
    A, B, al = value(a, 0), value(b, 0), sa.double() * sb.double()
    z = A @ B.t() * al
    want = z * (pre.double() > 0) if grad else z.clamp_min(0) + pre.double()
    tol = (k + 8) * 2.0 ** -23 * (A.abs() @ B.abs().t() * al) + 2.0 ** -8 * want.abs() + 1e-6
    return out, want, tol


@pytest.mark.parametrize("m,n,k,grad", [(2048, 2560, 16384, False), (128, 256, 65536, False),
                                        (2048, 2560, 16384, True), (128, 256, 65536, True)])
def test_expired_wait_is_reported_and_the_context_stays_usable(m, n, k, grad):
    """With the wait bound at zero a wait of the kernel runs out: the call ends,
    the status says so, and the next call is right (CTA pairs; one CTA per
    tile, with K split over a cluster in the forward epilogue)."""
    F = lib()
    assert F.fp8_get_last_device_error()[0] == 0
    F.fp8_set_option(F.OPT_WAIT_LIMIT_US, 0)
    try:
        run_plain_epilogue(m, n, k, grad)
        torch.cuda.synchronize()
    finally:
        F.fp8_set_option(F.OPT_WAIT_LIMIT_US, 2_000_000)
    assert F.fp8_get_last_device_error()[0] == F.FP8_ERR_TIMEOUT
    close(*run_plain_epilogue(m, n, k, grad))
    assert F.fp8_get_last_device_error() == (0, 0)


@pytest.mark.parametrize("m,n,k", [(1029, 1283, 272), (2048, 2560, 160)])
@pytest.mark.parametrize("grad", [False, True])
def test_without_cta_pairs(m, n, k, grad):
    """The same shapes on one CTA per tile."""
    F = lib()
    F.fp8_set_option(F.OPT_GEMM_CTA_PAIRS, 0)
    try:
        close(*run_plain_epilogue(m, n, k, grad))
    finally:
        F.fp8_set_option(F.OPT_GEMM_CTA_PAIRS, 1)


def test_group_without_multicast():
    F = lib()
    a, sa, b, sb, A, B = group_operands(2200, 2600, 384, 1)
    outs = []
    for on in (0, 1):
        F.fp8_set_option(F.OPT_GEMM_MULTICAST, on)
        outs.append(torch.empty((2200, 2600), dtype=torch.bfloat16, device="cuda"))
        F.fp8_gemm_group_epilogue(a, sa, b, sb, 1, outs[-1], act=F.ACT_SILU)
    assert torch.equal(*outs)


def test_repeatable():
    """Maxima, column sums and codes have the same bits on every run."""
    F = lib()
    m, n, k = 1500, 2576, 528
    a, sa = codes(randn(m, k), 1)
    b, sb = codes(randn(k, n, seed=1), 0)
    pre = randn(m, n, seed=2).bfloat16()
    got = []
    for _ in range(3):
        q = torch.empty((m, n), dtype=torch.uint8, device="cuda")
        am, db = torch.empty(1, device="cuda"), torch.empty(n, device="cuda")
        F.fp8_gemm_tensor_act_backward(a, 1, b, 0, sa, sb, pre, F.ACT_SILU, q=q,
                                       q_scale=torch.full((1,), 0.01, device="cuda"), q_amax=am,
                                       dbias=db, b_layout=F.MN_MAJOR)
        got.append((q, am, db))
    for g in got[1:]:
        assert all(torch.equal(x, y) for x, y in zip(got[0], g))


def test_own_scratch_on_two_streams():
    """Calls without a workspace on two streams at once: neither sees the
    other's partial sums."""
    F = lib()
    m, n, k = 300, 1040, 528
    a, sa = codes(randn(m, k), 0)
    pre = randn(m, n, seed=2).bfloat16()
    streams = [torch.cuda.Stream() for _ in range(2)]
    bs, dbs = [], []
    for i in range(2):
        b, sb = codes(randn(n, k, seed=10 + i), 0)
        bs.append((b, sb))
        dbs.append([torch.empty(n, device="cuda") for _ in range(20)])
    for st in streams:
        st.wait_stream(torch.cuda.current_stream())
    for j in range(20):
        for i, st in enumerate(streams):
            with torch.cuda.stream(st):
                F.fp8_gemm_tensor_act_backward(a, 0, bs[i][0], 0, sa, bs[i][1], pre, F.ACT_GELU,
                                               q=torch.empty((m, n), dtype=torch.uint8, device="cuda"),
                                               q_scale=sa, dbias=dbs[i][j])
    torch.cuda.synchronize()
    for i in range(2):
        want = torch.empty(n, device="cuda")
        ws = torch.empty(F.fp8_act_backward_workspace(m, n), dtype=torch.uint8, device="cuda")
        F.fp8_gemm_tensor_act_backward(a, 0, bs[i][0], 0, sa, bs[i][1], pre, F.ACT_GELU,
                                       out=torch.empty((m, n), device="cuda"), dbias=want, workspace=ws)
        assert all(torch.equal(d, want) for d in dbs[i])


@pytest.mark.parametrize("kind", ["tensor", "mx", "f32", "grad"])
def test_long_output_offsets(kind):
    """Outputs, residual, pre and codes whose element offsets pass 2^31: the
    last rows, the only ones with operands other than zero."""
    F = lib()
    m, n, k, t = 66049, 32784, 128, 200
    x = torch.zeros((m, k), device="cuda")
    x[-t:] = randn(t, k)
    if kind in ("mx", "f32"):
        a, sa, b, sb, A, B = group_operands(m, n, k, int(kind == "mx"))
        A, al, rows = A[-t:], 1.0, slice(m - t, m)
    else:
        a, sa = codes(x, 0)
        b, sb = codes(randn(n, k, seed=1), 0)
        A, B, al, rows = value(a, 0)[-t:], value(b, 0), sa.double() * sb.double(), slice(m - t, m)
    other = torch.zeros((m, n), dtype=torch.bfloat16, device="cuda")  # residual, or pre
    other[rows] = randn(t, n, seed=2).bfloat16()
    o = other[rows].double()
    z = A @ B.t() * al
    tz = (k + 8) * 2.0 ** -23 * (A.abs() @ B.abs().t() * al)
    c = torch.empty((m, n), dtype=torch.bfloat16, device="cuda")
    q = torch.empty((m, n), dtype=torch.uint8, device="cuda")
    qs, am = torch.full((1,), 0.1, device="cuda"), torch.empty(1, device="cuda")
    if kind == "grad":
        db = torch.empty(n, device="cuda")
        F.fp8_gemm_tensor_act_backward(a, 0, b, 0, sa, sb, other, F.ACT_SILU, out=c, q=q,
                                       q_fmt=F.E4M3, q_scale=qs, q_amax=am, dbias=db)
        s = act64(o, "silu")[1]
        y, ty = z * s, tz * s.abs() + 2.0 ** -18 * z.abs() * (1 + s.abs()) + 1e-30
        close(c[rows], y, ty + 2.0 ** -8 * (y.abs() + ty))
        sq = qs.double()
        v = (y / sq).clamp(-448, 448)
        err = (value(q[rows], 0) - v).abs()
        assert (err <= half_step(v.abs() + ty / sq, 0) * (1 + 1e-6) + 2 * ty / sq).all()
        close(db, y.sum(0), ty.sum(0) + (m // 32 + 32) * 2.0 ** -24 * y.abs().sum(0))
    else:
        p = torch.empty((m, n), dtype=torch.bfloat16, device="cuda")
        if kind == "tensor":
            F.fp8_gemm_tensor_epilogue(a, 0, b, 0, sa, sb, c, act=F.ACT_RELU, residual=other,
                                       pre_out=p, q=q, q_scale=qs, q_amax=am)
        else:
            F.fp8_gemm_group_epilogue(a, sa, b, sb, int(kind == "mx"), c, act=F.ACT_RELU,
                                      residual=other, pre_out=p)
        y = z.clamp_min(0) + o
        check_epilogue(None, y, tz + 2.0 ** -23 * o.abs(), z, "relu", c[rows], p[rows],
                       q[rows] if kind == "tensor" else None, qs, am, 0)
        if kind == "tensor":
            assert (q[:-t] == 0).all() and (c[:-t] == 0).all()
    assert F.fp8_get_last_device_error() == (0, 0)


def test_short_scales_are_refused():
    """Scale tensors of too few elements or of the other format's size."""
    F = lib()
    m, n, k = 40, 200, 384
    a, sa, b, sb, _, _ = group_operands(m, n, k, 0)
    c = torch.empty((m, n), dtype=torch.bfloat16, device="cuda")
    byte = torch.zeros(sa.numel(), dtype=torch.uint8, device="cuda")
    for s, t in ((sa.flatten()[:-1], sb), (sa, sb.flatten()[:-1]), (byte, sb), (sa.double(), sb)):
        with pytest.raises(ValueError):
            F.fp8_gemm_group_epilogue(a, s, b, t, F.SCALE_F32, c)
    with pytest.raises(ValueError):
        F.fp8_gemm_group_epilogue(a, sa, b, sb, F.SCALE_UE8M0, c)
    x, q = randn(m, k).bfloat16(), torch.empty((m, k), dtype=torch.uint8, device="cuda")
    for kw in (dict(scales=sa.flatten()[:-1]), dict(scales=byte), dict(scales=sa, sfmt=F.SCALE_UE8M0),
               dict(local=torch.zeros(k // 128 * 128 - 1, dtype=torch.int32, device="cuda"))):
        with pytest.raises(ValueError):
            F.fp8_rmsnorm_quantize(x, None, 1e-5, F.E4M3, q, **kw)
