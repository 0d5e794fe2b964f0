"""Tokens to their experts' rows and back, against the definitions in 64 bits
(plain torch, none of the library's code).

Tolerances.  combine: an fp32 chain of at most S fused steps and the residual's
addition, each within 2^-24 of a partial sum that is at most the sum of the
magnitudes; the result is rounded once to the output's type (half a step).
dw: a lane adds four pairs per 256 columns and a CTA has at least four warps up
to K = 16384 (16 windows each: 64 steps), then two halves, five shuffles and at
most eight warps: 80 steps of 2^-24 on the sum of the magnitudes cover it.  (One
warp alone: four pairs of each 256 columns too, 20 steps up to K = 1040, and the
same end.)  Codes of w dy: one rounding each
of the product, the maximum's product, the scale, its reciprocal and the
quotient, below 2^-21 together, and half a step of the format.  gather forms the
exact quotient: the bytes themselves are checked.
"""
import math

import pytest
import torch

from gpu_util import lib

pytestmark = pytest.mark.gpu

F8 = (torch.float8_e4m3fn, torch.float8_e5m2)
TOP = (448.0, 57344.0)
MANT, EMIN = (3, 2), (-6, -14)  # mantissa bits, exponent of the smallest normal
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
FILL = 0xA5


def choices(t, s, e, seed, drop=0.0, dtype=torch.int64):
    g = torch.Generator(device="cuda").manual_seed(seed)
    ids = torch.randint(0, e, (t, s), generator=g, device="cuda")
    if drop:
        u = torch.rand((t, s), generator=g, device="cuda")
        ids = torch.where(u < drop / 2, -1, torch.where(u > 1 - drop / 2, ids + e, ids))
    return ids.to(dtype)


def order(ids, e):
    """offsets, rows, pairs by a stable sort."""
    flat = ids.reshape(-1).long()
    kept = (flat >= 0) & (flat < e)
    key = torch.where(kept, flat, e)
    by = torch.argsort(key, stable=True)
    rows = torch.empty_like(by)
    rows[by] = torch.arange(by.numel(), device="cuda")
    count = torch.bincount(key, minlength=e + 1)[:e]
    offsets = torch.cat([count.new_zeros(1), count.cumsum(0)])
    n = int(offsets[-1])
    pairs = torch.where(torch.arange(by.numel(), device="cuda") < n, by, -1)
    return (offsets.int(), torch.where(kept, rows, -1).int().view(ids.shape), pairs.int())


def randn(shape, dtype, seed, std=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda") * std).to(dtype)


def pitched(t, pad):
    if not pad:
        return t.contiguous()
    wide = torch.full((t.shape[0], t.shape[1] + pad), 3.0, dtype=t.dtype, device=t.device)
    wide[:, :t.shape[1]] = t
    return wide[:, :t.shape[1]]


def filled(shape, dtype):
    return torch.full(shape, FILL if dtype == torch.uint8 else -7.0, dtype=dtype, device="cuda")


# ------------------------------------------------------------------- sort --

def run_sort(ids, e, pairs=True):
    F = lib()
    t, s = ids.shape
    offsets = torch.full((e + 1,), -5, dtype=torch.int32, device="cuda")
    rows = torch.full((t, s), -5, dtype=torch.int32, device="cuda")
    pr = torch.full((t * s,), -5, dtype=torch.int32, device="cuda") if pairs else None
    F.fp8_experts_sort(ids, e, offsets, rows, pr)
    return offsets, rows, pr


@pytest.mark.parametrize("t,s,e,drop,dtype", [
    (1, 1, 1, 0, torch.int64), (1, 8, 256, 0, torch.int32), (5, 3, 7, 0.5, torch.int64),
    (31, 1, 2, 0, torch.int32), (32, 1, 256, 0, torch.int64), (33, 1, 33, 0.3, torch.int32),
    (512, 8, 256, 0, torch.int64), (4097, 1, 5, 0, torch.int32),      # the two launch shapes
    (1366, 3, 255, 0.2, torch.int64), (16384, 8, 256, 0.25, torch.int32),
    (16411, 7, 64, 0, torch.int64), (100003, 10, 31, 0.1, torch.int32)])
def test_sort(t, s, e, drop, dtype):
    ids = choices(t, s, e, t + s + e, drop, dtype)
    want = order(ids, e)
    for got in (run_sort(ids, e), run_sort(ids, e)):
        for a, b in zip(got, want):
            assert torch.equal(a, b)
    offsets, rows, _ = run_sort(ids, e, pairs=False)
    assert torch.equal(offsets, want[0]) and torch.equal(rows, want[1])


@pytest.mark.parametrize("t,s", [(64, 8), (3000, 5)])
def test_sort_one_expert_or_none(t, s):
    ids = torch.full((t, s), 3, dtype=torch.int32, device="cuda")
    offsets, rows, pairs = run_sort(ids, 6)
    assert offsets.tolist() == [0, 0, 0, 0] + [t * s] * 3
    at = torch.arange(t * s, dtype=torch.int32, device="cuda")
    assert torch.equal(rows.view(-1), at) and torch.equal(pairs, at)
    for bad in (-1, 6, 2 ** 31 - 1, -2 ** 31):
        offsets, rows, pairs = run_sort(torch.full_like(ids, bad), 6)
        assert (offsets == 0).all() and (rows == -1).all() and (pairs == -1).all()
    wide = torch.full((t, s), (1 << 32) + 3, dtype=torch.int64, device="cuda")
    assert (run_sort(wide, 6)[1] == -1).all()


def test_sort_no_tokens():
    offsets, _, _ = run_sort(torch.empty((0, 4), dtype=torch.int64, device="cuda"), 9)
    assert (offsets == 0).all()


# ----------------------------------------------------------------- gather --

def quotient(x, y):
    """fl32(x / y) (torch multiplies by the rounded reciprocal of a scalar)."""
    return x / torch.full_like(x, y)


def group_codes(x, sfmt, fmt):
    """Codes and scales as fp8_quantize_token_group defines them, in torch."""
    m, k = x.shape
    g = (k + 127) // 128
    xp = torch.nn.functional.pad(x.float(), (0, g * 128 - k)).view(m, g, 128)
    top = xp.abs().amax(2)
    s = torch.where(top > 0, quotient(top, TOP[fmt]), torch.ones_like(top))
    if sfmt:
        man, e = torch.frexp(s)
        e = torch.where(man == 0.5, e - 1, e)
        s, kept = torch.ldexp(torch.ones_like(s), e), (e + 127).to(torch.uint8)
    else:
        kept = s
    q = (xp / s.unsqueeze(2)).clamp(-TOP[fmt], TOP[fmt]).to(F8[fmt])
    return q.view(m, g * 128)[:, :k].contiguous().view(torch.uint8), kept.t().contiguous()


GATHER = [  # t, s, e, k, dt, sfmt, fmt, drop, pad, spare rows
    (1, 1, 1, 16, "bf16", 0, 0, 0, 0, 0), (1, 8, 256, 7168, "bf16", 0, 0, 0, 0, 0),
    (3, 2, 4, 128, "f32", 1, 0, 0, 0, 5), (64, 8, 256, 2064, "bf16", 1, 1, 0.3, 8, 0),
    (77, 3, 5, 144, "f32", 0, 1, 0.5, 24, 40), (257, 6, 16, 1040, "bf16", 0, 0, 0.2, 0, 3),
    (9, 33, 40, 640, "bf16", 0, 0, 0.1, 0, 0), (5, 70, 70, 528, "f32", 1, 0, 0, 0, 0),
    (1500, 8, 64, 4096, "bf16", 0, 0, 0, 0, 0), (4, 2, 2, 20480, "f32", 0, 0, 0, 0, 0),
    # short lists of many tokens, of which two windows of columns go at once
    (4100, 2, 8, 1040, "bf16", 0, 0, 0.1, 8, 3), (3100, 4, 16, 1296, "f32", 1, 1, 0.2, 0, 0),
    (7000, 1, 8, 528, "bf16", 1, 1, 0, 0, 0)]


@pytest.mark.parametrize("t,s,e,k,dt,sfmt,fmt,drop,pad,spare", GATHER)
def test_gather(t, s, e, k, dt, sfmt, fmt, drop, pad, spare):
    F = lib()
    _, rows, _ = order(choices(t, s, e, t + k, drop), e)
    x = randn((t, k), DT[dt], 1, 2.0)
    x[:, ::97] *= 30
    x[0, :k // 2] = 0  # groups of zeros
    m, g = t * s + spare, (k + 127) // 128
    st = torch.uint8 if sfmt else torch.float32
    q, sc = filled((m, k), torch.uint8), filled((g, m), st)
    out = filled((m, k), DT[dt])
    F.fp8_experts_gather(pitched(x, pad), rows, q=q, scales=sc, fmt=fmt, sfmt=sfmt, out=out)
    tq, ts = group_codes(x, sfmt, fmt)
    wq, wsc, wout = filled((m, k), torch.uint8), filled((g, m), st), filled((m, k), DT[dt])
    pair = torch.nonzero(rows.reshape(-1) >= 0).squeeze(1)
    at, tok = rows.reshape(-1)[pair].long(), pair // s
    wq[at], wout[at] = tq[tok], x[tok]
    wsc[:, at] = ts[:, tok]
    assert torch.equal(sc, wsc) and torch.equal(q, wq) and torch.equal(out, wout)
    # the library's own quantizer gives the same codes
    lq, ls = torch.empty_like(tq), torch.empty_like(ts)
    F.fp8_quantize_token_group(x, fmt, sfmt, lq, ls)
    assert torch.equal(lq, tq) and torch.equal(ls, ts)
    # codes that exist already are moved
    q2, sc2 = filled((m, k), torch.uint8), filled((g, m), st)
    F.fp8_experts_gather(tq, rows, q=q2, scales=sc2, fmt=fmt, sfmt=sfmt, x_scales=ts)
    assert torch.equal(q2, wq) and torch.equal(sc2, wsc)
    # the rows alone
    out2 = filled((m, k), DT[dt])
    F.fp8_experts_gather(pitched(x, pad), rows, out=out2)
    assert torch.equal(out2, wout)


def test_gather_non_finite():
    """As the quantizer: a NaN stays one beside values under a scale of 1, a
    group with an infinity becomes zeros and NaN."""
    F = lib()
    x = randn((4, 256), torch.bfloat16, 5)
    x[0, 3], x[1, 130], x[2, 0], x[3, 255] = float("nan"), float("inf"), -float("inf"), 3e38
    rows = torch.tensor([[2], [0], [3], [1]], dtype=torch.int32, device="cuda")
    for sfmt, st in ((0, torch.float32), (1, torch.uint8)):
        q, sc = filled((4, 256), torch.uint8), filled((2, 4), st)
        F.fp8_experts_gather(x, rows, q=q, scales=sc, sfmt=sfmt)
        lq, ls = torch.empty_like(q), torch.empty_like(sc)
        F.fp8_quantize_token_group(x, 0, sfmt, lq, ls)
        at = rows.view(-1).long()
        nan = (lq & 0x7F) == 0x7F
        assert torch.equal(((q[at] & 0x7F) == 0x7F), nan)
        assert torch.equal(q[at][~nan], lq[~nan])
        assert torch.equal(sc[:, at].contiguous().view(torch.uint8), ls.view(torch.uint8))


@pytest.mark.parametrize("s,dt", [(1, "bf16"), (8, "f32")])
def test_gather_extreme_scales(s, dt):
    """Rows from 2^-120 to 2^120 among others: the quantizer's bytes."""
    F = lib()
    t, k = 7000, 528
    x = randn((t, k), torch.float32, 5)
    x *= torch.exp2(torch.arange(t, device="cuda") % 241 - 120.0)[:, None]
    x = x.to(DT[dt])
    rows = torch.randperm(t * s, device="cuda").int().view(t, s)
    for fmt in (0, 1):
        for sfmt, st in ((0, torch.float32), (1, torch.uint8)):
            q, sc = filled((t * s, k), torch.uint8), filled((5, t * s), st)
            F.fp8_experts_gather(x, rows, q=q, scales=sc, fmt=fmt, sfmt=sfmt)
            lq, ls = torch.empty((t, k), dtype=torch.uint8, device="cuda"), filled((5, t), st)
            F.fp8_quantize_token_group(x, fmt, sfmt, lq, ls)
            for j in range(s):
                at = rows[:, j].long()
                assert torch.equal(q[at], lq) and torch.equal(sc[:, at], ls)


# ---------------------------------------------------------------- combine --

COMBINE = [  # t, s, e, k, dt, out, res, weights, drop, pad
    (1, 1, 1, 16, "bf16", "bf16", False, True, 0, 0), (1, 8, 256, 7168, "bf16", "bf16", True, True, 0, 0),
    (63, 2, 8, 256, "f32", "f32", True, False, 0.4, 8), (40, 9, 16, 1040, "bf16", "f32", False, True, 0.3, 16),
    (7, 33, 64, 144, "f32", "bf16", True, True, 0.2, 0), (300, 6, 32, 2064, "bf16", "bf16", True, False, 0, 24),
    (3, 70, 70, 528, "bf16", "bf16", False, True, 0.9, 0), (1500, 8, 64, 4096, "bf16", "bf16", True, True, 0, 0),
    # short lists, of which several windows of columns go at once
    (90, 2, 8, 2064, "bf16", "bf16", True, True, 0.2, 8), (33, 1, 4, 1040, "bf16", "f32", True, False, 0, 0),
    (50, 3, 5, 1296, "bf16", "bf16", False, True, 0.3, 0), (700, 4, 9, 4112, "bf16", "f32", True, True, 0.1, 16),
    (41, 2, 8, 1040, "f32", "bf16", True, True, 0.2, 0), (300, 1, 8, 7168, "f32", "f32", False, True, 0, 8)]


@pytest.mark.parametrize("t,s,e,k,dt,odt,res,weights,drop,pad", COMBINE)
def test_combine(t, s, e, k, dt, odt, res, weights, drop, pad):
    F = lib()
    _, rows, _ = order(choices(t, s, e, 3 * t + k, drop), e)
    m = t * s + 2
    x = randn((m, k), DT[dt], 2)
    owned = torch.zeros(m, dtype=torch.bool, device="cuda")
    owned[rows[rows >= 0].long()] = True
    x[~owned] = float("nan")  # rows that no pair owns are not read
    w = torch.softmax(randn((t, s), torch.float32, 3), 1) if weights else None
    if weights:
        w = torch.where(rows < 0, float("nan"), w)  # nor are dropped pairs' weights
    r = randn((t, k), DT[odt], 4, 3.0) if res else None
    out = filled((t, k + pad), DT[odt])
    F.fp8_experts_combine(pitched(x, pad), rows, w, out[:, :k], residual=None if r is None else pitched(r, pad))
    kept = (rows >= 0)
    picked = torch.where(kept[:, :, None], x[rows.clamp_min(0).long()].double(), 0.0)
    wd = torch.where(kept, w.double(), 0.0) if weights else kept.double()
    terms = picked * wd[:, :, None]
    want, mag = terms.sum(1), terms.abs().sum(1)
    if res:
        want, mag = want + r.double(), mag + r.double().abs()
    err = (out[:, :k].double() - want).abs()
    tol = (s + 1) * 2.0 ** -24 * mag * (1 + 2.0 ** -7)
    tol = tol + HALF[DT[odt]] * (want.abs() + tol) + 1e-40
    assert (err <= tol).all(), float((err - tol).max())
    assert (out[:, k:] == -7.0).all()  # the columns behind the rows
    if res:  # in place
        acc = pitched(r, pad)
        F.fp8_experts_combine(pitched(x, pad), rows, w, acc, residual=acc)
        assert torch.equal(acc, out[:, :k])


def test_combine_without_a_kept_pair():
    F = lib()
    rows = torch.tensor([[-1, 99], [-3, 8]], dtype=torch.int32, device="cuda")  # 8 is M itself
    x = randn((8, 256), torch.bfloat16, 1)
    r = randn((2, 256), torch.bfloat16, 2)
    out = torch.empty_like(r)
    F.fp8_experts_combine(x, rows, None, out, residual=r)
    assert torch.equal(out, r)
    F.fp8_experts_combine(x, rows, None, out)
    assert (out == 0).all()
    F.fp8_experts_combine(x[:0], rows, None, out, residual=r)  # no rows at all
    assert torch.equal(out, r)


# ------------------------------------------------------- combine, gradient --

def half_step(v, fmt):
    e = torch.floor(torch.log2(v.abs().clamp_min(2.0 ** EMIN[fmt])))
    return torch.exp2(e - MANT[fmt] - 1)


REL = 2.0 ** -21

GRAD = [  # t, s, e, k, dt, dydt, sfmt, fmt, dw, weights, drop, pad
    (1, 1, 1, 16, "bf16", "bf16", 0, 0, True, True, 0, 0), (1, 8, 256, 7168, "bf16", "bf16", 0, 0, True, True, 0, 0),
    (19, 2, 8, 2064, "f32", "f32", 0, 1, True, True, 0.3, 8), (50, 9, 16, 144, "bf16", "f32", 1, 0, True, True, 0.3, 0),
    (7, 33, 64, 528, "f32", "bf16", 0, 0, True, False, 0.2, 16), (300, 6, 32, 1040, "bf16", "bf16", 1, 1, False, True, 0, 0),
    (3, 70, 70, 640, "bf16", "bf16", 0, 0, True, True, 0.8, 0), (800, 8, 64, 4096, "bf16", "bf16", 0, 0, True, True, 0, 0),
    (5, 4, 8, 16384, "bf16", "f32", 0, 0, True, True, 0, 0),
    # short lists, of which several windows of columns go at once
    (90, 2, 8, 2064, "bf16", "bf16", 0, 0, True, True, 0.2, 8), (33, 1, 4, 1040, "bf16", "f32", 1, 1, True, False, 0, 0),
    (50, 3, 5, 1296, "bf16", "bf16", 0, 1, True, True, 0.3, 0), (700, 4, 9, 4112, "bf16", "f32", 0, 0, True, True, 0.1, 16),
    (300, 1, 8, 7168, "f32", "bf16", 0, 0, True, True, 0, 8), (64, 2, 8, 16384, "bf16", "bf16", 0, 0, True, True, 0, 0),
    # many tokens, of which a warp takes one alone
    (16000, 2, 8, 528, "bf16", "bf16", 0, 0, True, True, 0.1, 0), (15001, 9, 16, 144, "bf16", "f32", 1, 0, True, True, 0.2, 0),
    (12000, 1, 8, 1040, "f32", "f32", 0, 1, True, False, 0, 8)]


@pytest.mark.parametrize("t,s,e,k,dt,dydt,sfmt,fmt,dw,weights,drop,pad", GRAD)
def test_combine_backward(t, s, e, k, dt, dydt, sfmt, fmt, dw, weights, drop, pad):
    F = lib()
    _, rows, _ = order(choices(t, s, e, 5 * t + k, drop), e)
    m, g = t * s + 3, (k + 127) // 128
    dy = randn((t, k), DT[dydt], 1, 1e-3)
    dy[0, :k // 2] = 0
    x = randn((m, k), DT[dt], 2)
    w = randn((t, s), torch.float32, 3, 0.5) if weights else None  # of both signs
    st = torch.uint8 if sfmt else torch.float32

    def run(codes=True, rows_out=None):
        q, sc = (filled((m, k), torch.uint8), filled((g, m), st)) if codes else (None, None)
        dx = filled((m, k + pad), rows_out) if rows_out is not None else None
        dwv = filled((t, s), torch.float32) if dw else None
        F.fp8_experts_combine_backward(
            pitched(dy, pad), rows, w, x=pitched(x, pad) if dw else None, d_weights=dwv, q=q,
            scales=sc, fmt=fmt, sfmt=sfmt, dx=None if dx is None else dx[:, :k])
        return q, sc, dx, dwv

    q, sc, dx, dwv = run(rows_out=torch.bfloat16)
    pair = torch.nonzero(rows.reshape(-1) >= 0).squeeze(1)
    at, tok = rows.reshape(-1)[pair].long(), pair // s
    wp = w.reshape(-1)[pair].double() if weights else torch.ones(pair.numel(), dtype=torch.float64, device="cuda")
    v = dy.double()[tok] * wp[:, None]
    # scales
    vp = torch.nn.functional.pad(v, (0, g * 128 - k)).view(-1, g, 128)
    top = vp.abs().amax(2)
    got = sc[:, at].t()
    want = torch.where(top > 0, top / TOP[fmt], torch.ones_like(top))
    if sfmt:
        ge = torch.exp2(got.double() - 127)
        ok = (ge >= want * (1 - REL)) & (ge / 2 < want * (1 + REL))
        assert (ok | ((top == 0) & (got == 127))).all()
    else:
        ge = got.double()
        assert ((ge - want).abs() <= REL * want).all()
    # codes, under the scales as stored
    u = (vp / ge[:, :, None]).view(-1, g * 128)[:, :k].clamp(-TOP[fmt], TOP[fmt])
    err = (q[at].view(F8[fmt]).double() - u).abs()
    assert (err <= half_step(u, fmt) * (1 + 1e-6) + REL * u.abs()).all()
    # rows in bf16, and in fp32
    assert ((dx[at, :k].double() - v).abs() <= (2.0 ** -8 + 2.0 ** -23) * v.abs() + 1e-40).all()
    dx32 = run(codes=False, rows_out=torch.float32)[2]
    assert ((dx32[at, :k].double() - v).abs() <= 2.0 ** -24 * v.abs() + 1e-44).all()
    # nothing else was written
    other = torch.ones(m, dtype=torch.bool, device="cuda")
    other[at] = False
    assert (q[other] == FILL).all() and (dx[other] == -7.0).all() and (dx[:, k:] == -7.0).all()
    assert (sc[:, other] == (FILL if sfmt else -7.0)).all()
    if dw:
        want = torch.zeros(t * s, dtype=torch.float64, device="cuda")
        mag = torch.zeros_like(want)
        prod = dy.double()[tok] * x.double()[at]
        want[pair], mag[pair] = prod.sum(1), prod.abs().sum(1)
        assert ((dwv.double().view(-1) - want).abs() <= 80 * 2.0 ** -24 * mag + 1e-40).all()
        alone = torch.empty_like(dwv)
        F.fp8_experts_combine_backward(pitched(dy, pad), rows, w, x=pitched(x, pad), d_weights=alone)
        assert torch.equal(alone, dwv)
    again = run(rows_out=torch.bfloat16)
    for a, b in zip((q, sc, dx, dwv), again):
        assert a is None or torch.equal(a, b)


def test_combine_backward_extreme_scales():
    """Weights that make the groups' scales leave the range of the rounded
    reciprocal (IEEE division there), and a weight of zero."""
    F = lib()
    k = 256
    dy = randn((4, k), torch.float32, 1)
    w = torch.tensor([[1e-37], [3e37], [0.0], [-1.0]], device="cuda")
    rows = torch.arange(4, dtype=torch.int32, device="cuda").view(4, 1)
    q, sc = filled((4, k), torch.uint8), filled((2, 4), torch.float32)
    F.fp8_experts_combine_backward(dy, rows, w, q=q, scales=sc)
    v = (dy * w)  # the fp32 products, as the kernel forms them
    top = v.view(4, 2, 128).abs().amax(2)
    want = torch.where(top > 0, quotient(top, 448.0), torch.ones_like(top))
    assert torch.equal(sc.t(), want)
    u = (v.double().view(4, 2, 128) / want.double()[:, :, None]).view(4, k)
    err = (q.view(F8[0]).double() - u).abs()
    assert (err <= half_step(u, 0) * (1 + 1e-6) + REL * u.abs()).all()


@pytest.mark.parametrize("s,dt", [(2, torch.bfloat16), (5, torch.float32), (11, torch.bfloat16)])
def test_dropped_pairs_beside_non_finite_gradients(s, dt):
    """A dropped pair's dw is 0 whatever dy holds, and its neighbours' are the sums."""
    F = lib()
    t, k = 6, 528
    ids = choices(t, s, 4, s, 0.4)
    _, rows, _ = order(ids, 4)
    x, dy = randn((t * s, k), dt, 1), randn((t, k), dt, 2)
    dy[0, 3], dy[1, 300], dy[2, 527], dy[3] = math.inf, -math.inf, math.nan, math.inf
    dw = filled((t, s), torch.float32)
    F.fp8_experts_combine_backward(dy, rows, torch.ones((t, s), device="cuda"), x=x, d_weights=dw)
    gone = rows < 0
    assert gone.any() and (dw[gone] == 0).all()
    assert not dw[:4][~gone[:4]].isfinite().any()
    want = (dy.double()[:, None] * x.double()[rows.clamp_min(0).long()]).sum(2)
    size = (dy.double()[:, None] * x.double()[rows.clamp_min(0).long()]).abs().sum(2)
    ok = (dw.double() - want).abs() <= 80 * 2.0 ** -24 * size
    assert ok[4:][~gone[4:]].all()


def test_gather_is_the_transpose_of_combine():
    """<combine(x), dy> = <x, rows of combine_backward(dy)> and the same for
    gather: the gradients against differences (the maps are linear: a
    difference is the map itself), up to the fp32 sums."""
    F = lib()
    t, s, e, k = 37, 4, 6, 144
    _, rows, _ = order(choices(t, s, e, 1, 0.3), e)
    m = t * s
    x, dy = randn((m, k), torch.float32, 1), randn((t, k), torch.float32, 2)
    w = randn((t, s), torch.float32, 3)
    y, dx = torch.empty((t, k), device="cuda"), torch.zeros((m, k), device="cuda")
    dw = torch.empty((t, s), device="cuda")
    F.fp8_experts_combine(x, rows, w, y)
    F.fp8_experts_combine_backward(dy, rows, w, x=x, d_weights=dw, dx=dx)
    a, b = (y.double() * dy.double()).sum(), (dx.double() * x.double()).sum()
    c = (dw.double() * torch.where(rows < 0, 0.0, w).double()).sum()
    mag = float((y.abs().double() * dy.abs().double()).sum()) * 16
    assert abs(float(a - b)) <= 2.0 ** -20 * mag and abs(float(a - c)) <= 2.0 ** -20 * mag
    xt, back = randn((t, k), torch.float32, 4), torch.empty((t, k), device="cuda")
    grouped = torch.zeros((m, k), device="cuda")
    F.fp8_experts_gather(xt, rows, out=grouped)
    F.fp8_experts_combine(x, rows, None, back)
    a, b = (grouped.double() * x.double()).sum(), (back.double() * xt.double()).sum()
    assert abs(float(a - b)) <= 2.0 ** -20 * float((grouped.abs() * x.abs()).double().sum())


# -------------------------------------------------- addresses, streams, graphs --

def test_rows_beyond_32_bit_offsets():
    """Rows whose byte and element offsets pass 2^32."""
    F = lib()
    k, m = 16384, 270000
    x = randn((2, k), torch.bfloat16, 1)
    rows = torch.tensor([[m - 1, 5], [m - 2, 0]], dtype=torch.int32, device="cuda")
    q = torch.zeros((m, k), dtype=torch.uint8, device="cuda")
    sc = torch.zeros((k // 128, m), device="cuda")
    out = torch.zeros((m, k), dtype=torch.bfloat16, device="cuda")
    F.fp8_experts_gather(x, rows, q=q, scales=sc, out=out)
    tq, ts = group_codes(x, 0, 0)
    for t in range(2):
        for s in range(2):
            r = int(rows[t, s])
            assert torch.equal(q[r], tq[t]) and torch.equal(sc[:, r], ts[:, t])
            assert torch.equal(out[r], x[t])
    assert int((q != 0).any(1).sum()) == 4
    y = torch.empty_like(x)
    F.fp8_experts_combine(out, rows, None, y)
    assert torch.equal(y, (x.float() * 2).to(torch.bfloat16))
    dw = torch.empty((2, 2), device="cuda")
    F.fp8_experts_combine_backward(x, rows, None, x=out, d_weights=dw, q=q, scales=sc)
    want = (x.double() ** 2).sum(1)
    assert ((dw.double() - want[:, None]).abs() <= 80 * 2.0 ** -24 * want[:, None]).all()


def chain(F, ids, x, w, e, bufs):
    offsets, rows, q, sc, grouped, out, dw, dq, dsc = bufs
    F.fp8_experts_sort(ids, e, offsets, rows)
    F.fp8_experts_gather(x, rows, q=q, scales=sc, out=grouped)
    F.fp8_experts_combine(grouped, rows, w, out, residual=x)
    F.fp8_experts_combine_backward(out, rows, w, x=grouped, d_weights=dw, q=dq, scales=dsc)


def chain_buffers(t, s, e, k):
    m = t * s
    new = lambda *sh, dt=torch.float32: torch.zeros(*sh, dtype=dt, device="cuda")  # noqa: E731
    return (new(e + 1, dt=torch.int32), new(t, s, dt=torch.int32), new(m, k, dt=torch.uint8),
            new(k // 128, m), new(m, k, dt=torch.bfloat16), new(t, k, dt=torch.bfloat16),
            new(t, s), new(m, k, dt=torch.uint8), new(k // 128, m))


@pytest.mark.parametrize("t", [3, 700])
def test_captured_graphs_and_side_streams(t):
    """The chain captured once and replayed on new inputs equals direct calls;
    two graphs and a direct call on another stream do not disturb each other."""
    F = lib()
    s, e, k = 8, 64, 1024
    ids = [choices(t, s, e, i) for i in range(3)]
    xs = [randn((t, k), torch.bfloat16, 10 + i) for i in range(3)]
    ws = [randn((t, s), torch.float32, 20 + i) for i in range(3)]
    want = []
    for i in range(3):
        b = chain_buffers(t, s, e, k)
        chain(F, ids[i], xs[i], ws[i], e, b)
        want.append(b)
    torch.cuda.synchronize()
    graphs = []
    for i in range(2):
        b, ib, xb, wb = chain_buffers(t, s, e, k), ids[2].clone(), xs[2].clone(), ws[2].clone()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            chain(F, ib, xb, wb, e, b)
        ib.copy_(ids[i])
        xb.copy_(xs[i])
        wb.copy_(ws[i])
        graphs.append((g, b, ib, xb, wb))  # (a graph reads its inputs at every replay)
    torch.cuda.synchronize()
    side, other = torch.cuda.Stream(), torch.cuda.Stream()
    direct = chain_buffers(t, s, e, k)
    torch.cuda.synchronize()
    for _ in range(3):
        graphs[0][0].replay()
        with torch.cuda.stream(side):
            graphs[1][0].replay()
        with torch.cuda.stream(other):
            chain(F, ids[2], xs[2], ws[2], e, direct)
    torch.cuda.synchronize()
    for got, ref in zip((graphs[0][1], graphs[1][1], direct), want):
        for a, b in zip(got, ref):
            assert torch.equal(a, b)


FIRST = """
import torch
import fp8_quantized_gemm_gb300 as F
t, s, e, k = 700, 8, 256, 1024
ids = torch.randint(0, e, (t, s), device="cuda")
new = lambda *sh, dt=torch.float32: torch.zeros(*sh, dtype=dt, device="cuda")
x, w = torch.randn(t, k, device="cuda").bfloat16(), torch.rand(t, s, device="cuda")
off, rows, pairs = new(e + 1, dt=torch.int32), new(t, s, dt=torch.int32), new(t * s, dt=torch.int32)
q, sc, y = new(t * s, k, dt=torch.uint8), new(k // 128, t * s), new(t, k, dt=torch.bfloat16)
grouped, dw, hq = new(t * s, k, dt=torch.bfloat16), new(t, s), new(t, k, dt=torch.uint8)
hs, am, one = new(k // 128, t), new(1), torch.ones(1, device="cuda")
def run():
    F.fp8_experts_sort(ids, e, off, rows, pairs)
    F.fp8_experts_gather(x, rows, q=q, scales=sc, out=grouped)
    F.fp8_experts_combine(grouped, rows, w, y)
    F.fp8_experts_combine_backward(y, rows, w, x=grouped, d_weights=dw, q=q, scales=sc)
    F.fp8_act_checkpoint(x, None, F.ACT_SILU, hq, scale=one, amax_out=am)
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    run()
g.replay()
torch.cuda.synchronize()
got = [v.clone() for v in (off, rows, pairs, q, sc, y, dw, hq, am)]
run()
torch.cuda.synchronize()
assert all(torch.equal(a, b) for a, b in zip(got, (off, rows, pairs, q, sc, y, dw, hq, am)))
assert int(off[-1]) == t * s and float(am) > 0
print("fine")
"""


def test_first_calls_of_a_process_may_be_captured():
    """The kernels' attributes are set by their first launch."""
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", FIRST], cwd=root, capture_output=True, text=True,
                       timeout=300)
    assert r.returncode == 0 and "fine" in r.stdout, r.stderr[-2000:]


def test_binding_refuses():
    F = lib()
    t, s, e, k = 4, 2, 3, 256
    ids = choices(t, s, e, 1)
    offsets, rows, _ = run_sort(ids, e)
    x = randn((t, k), torch.bfloat16, 1)
    q, sc = torch.empty((8, k), dtype=torch.uint8, device="cuda"), torch.empty((2, 8), device="cuda")
    y, w = torch.empty_like(x), torch.ones((t, s), device="cuda")
    with pytest.raises(ValueError):
        F.fp8_experts_sort(ids.float(), e, offsets, rows)
    with pytest.raises(ValueError):
        F.fp8_experts_sort(ids, e + 1, offsets, rows)
    with pytest.raises(ValueError):
        F.fp8_experts_sort(ids.t(), e, offsets, rows)
    with pytest.raises(ValueError):
        F.fp8_experts_gather(x, rows, q=q)                       # scales missing
    with pytest.raises(ValueError):
        F.fp8_experts_gather(x, rows, q=q, scales=sc[:1])        # too few
    with pytest.raises(ValueError):
        F.fp8_experts_gather(x, rows)
    with pytest.raises(ValueError):
        F.fp8_experts_gather(x, rows.long(), q=q, scales=sc)
    with pytest.raises(ValueError):
        F.fp8_experts_gather(x, rows[:3], q=q, scales=sc)        # another T
    with pytest.raises(ValueError):
        F.fp8_experts_gather(x.half(), rows, q=q, scales=sc)
    with pytest.raises(ValueError):
        F.fp8_experts_combine(x, rows, w[:, :1], y)
    with pytest.raises(ValueError):
        F.fp8_experts_combine(x, rows, w, y, residual=x.float())
    with pytest.raises(ValueError):
        F.fp8_experts_combine(x.cpu(), rows, w, y)
    with pytest.raises(ValueError):
        F.fp8_experts_combine_backward(y, rows, w, d_weights=w)  # x missing
    with pytest.raises(ValueError):
        F.fp8_experts_combine_backward(y, rows, w, x=x[:, :128], d_weights=w)
    with pytest.raises(F.Fp8Error):
        F.fp8_experts_gather(x[:, :200], rows, out=torch.empty((8, 200), dtype=x.dtype, device="cuda"))
