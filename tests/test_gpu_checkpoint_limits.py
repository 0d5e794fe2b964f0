"""The checkpointed activation at the ends of its scales, in both scale formats:
tiny and huge groups, checkpoints of values beyond 2^49, infinities and NaN.

Tolerances are test_gpu_act_checkpoint.py's; what a group with an infinity or a NaN
holds is compared exactly.
"""
import math

import pytest
import torch

from gpu_util import lib
from test_gpu_act_checkpoint import (ACTS, BF, REL, TOP, check_group, check_kept, fill, groups, half_step,
                                     inputs, kept_values, quantizer, sdt, slope, value)

pytestmark = pytest.mark.gpu

SFMT = pytest.mark.parametrize("sfmt", [0, 1])


def check_codes(q, s, want, fmt, sfmt):
    """check_group for want that is exact in fp32, at scales down to the smallest: an
    FP32 scale of 1e-35 / 57344 = 6e-40 is subnormal, rounded to a multiple of 2^-149 and
    so off by up to 2^-150 beside its other roundings; a UE8M0 scale is not below 2^-127."""
    top = groups(want.abs()).amax(2)
    got = torch.exp2(s.t().double() - 127) if sfmt else s.t().double()
    ideal = top / TOP[fmt]
    if sfmt:
        ideal = ideal.clamp_min(2.0 ** -127)
        ok = (got >= ideal * (1 - 2.0 ** -22)) & (got / 2 < ideal * (1 + 2.0 ** -22))
        ok |= (got == 2.0 ** -127) & (ideal == got)
    else:
        ok = (got - ideal).abs() <= 2.0 ** -22 * ideal + 2.0 ** -150
    assert ok.all()
    u = (groups(want) / got[:, :, None]).flatten(1)[:, :want.shape[1]].clamp(-TOP[fmt], TOP[fmt])
    f8 = (torch.float8_e4m3fn, torch.float8_e5m2)[fmt]
    assert ((q.view(f8).double() - u).abs() <= half_step(u, fmt) * (1 + 1e-6) + 2.0 ** -22 * u.abs()).all()


@SFMT
@pytest.mark.parametrize("fmt", [0, 1])
def test_extreme_groups(sfmt, fmt):
    """Groups of 1e-35, 1 and 1e36 in one row and in one column."""
    F = lib()
    m, n = 6, 400
    by = torch.tensor([1e-35, 1.0, 1e36], device="cuda")
    which = (torch.arange(m, device="cuda")[:, None] + torch.arange(n, device="cuda") // 128) % 3
    h = (inputs(m, n, 4).float() * by[which]).to(BF)
    q, sc = fill((m, n), torch.uint8), fill((4, m), sdt(sfmt))
    hq, hs = fill((m, n), torch.uint8), fill((4, m), sdt(sfmt))
    F.fp8_act_checkpoint(h, None, F.ACT_NONE, q, scales=sc, fmt=fmt, sfmt=sfmt, keep_sfmt=sfmt, h_q=hq,
                         h_scales=hs)
    check_kept(hq, hs, h, sfmt)
    check_codes(q, sc, h.double(), fmt, sfmt)


def test_smallest_power_of_two_scale():
    """Groups below 448 x 2^-127 take the byte 0, and come back with it."""
    F = lib()
    n = 128
    h = (inputs(2, n, 5).float() * 2.0 ** -124).to(BF)
    q, sc = fill((2, n), torch.uint8), fill((1, 2), torch.uint8)
    hq, hs = fill((2, n), torch.uint8), fill((1, 2), torch.uint8)
    F.fp8_act_checkpoint(h, None, F.ACT_NONE, q, scales=sc, sfmt=1, keep_sfmt=1, h_q=hq, h_scales=hs)
    assert (sc == 0).all() and (hs == 0).all()
    want = (h.double() * 2.0 ** 127).float().to(torch.float8_e4m3fn).view(torch.uint8)
    assert torch.equal(q, want) and torch.equal(hq, want)
    # du = da h at the kept values: 2^120 x them, exact in fp32
    da = torch.full((2, n), 2.0 ** 120, dtype=BF, device="cuda")
    ones = torch.full((2, n), 0x38, dtype=torch.uint8, device="cuda")  # 1.0
    du = fill((2, n), BF)
    F.fp8_act_checkpoint_backward(da, F.ACT_NONE, hq, hs, ones, torch.full((1, 2), 127, dtype=torch.uint8, device="cuda"),
                                  keep_sfmt=1, du=du)
    assert torch.equal(du.double(), want.view(torch.float8_e4m3fn).double() * 2.0 ** -7)


@SFMT
@pytest.mark.parametrize("act,gate", [("silu", True), ("gelu_tanh", False), ("gelu", True)])
def test_checkpoints_of_large_values(act, gate, sfmt):
    """Checkpoints of about 1e15, where the slopes are 0 and 1, beside common ones."""
    F = lib()
    m, n = 40, 272
    h = inputs(m, n, 6).float()
    h[::3] *= 1e15
    h = h.to(BF)
    da, u = inputs(m, n, 7, 1e-3), inputs(m, n, 8) if gate else None
    kept, vals = {}, {}
    for name, x in (("h", h), ("u", u)):
        if x is not None:
            kept[name + "_q"], kept[name + "_scales"] = quantizer(x, sfmt)
            vals[name] = kept_values(kept[name + "_q"], kept[name + "_scales"], sfmt)
    out = {"d" + x: fill((m, n), BF) for x in vals}
    codes = {"d%s_q" % x: fill((m, n), torch.uint8) for x in vals}
    scales = {"d%s_scales" % x: fill((3, m), sdt(sfmt)) for x in vals}
    F.fp8_act_checkpoint_backward(da, ACTS.index(act), keep_sfmt=sfmt, sfmt=sfmt, fmt=0, **kept, **out,
                                  **codes, **scales)
    d, hv = da.double(), vals["h"]
    sl = slope(hv, act)
    want = {"dh": (d * sl, REL * d.abs() * sl.abs().clamp_min(1.0))}
    if gate:
        want = {"dh": (want["dh"][0] * vals["u"], want["dh"][1] * vals["u"].abs()),
                "du": (d * value(hv, act), REL * (d * value(hv, act)).abs())}
    for name, (w, e) in want.items():
        e = e + 1e-38
        assert ((out[name].double() - w).abs() <= 2.0 ** -8 * w.abs() + 2 * e).all()
        check_group(codes[name + "_q"], scales[name + "_scales"], w, e, 0, sfmt)


@SFMT
def test_a_group_with_an_infinity(sfmt):
    """FP32: the scale is infinite, the infinity a NaN code and the rest zeros: the
    group stands for NaN.  UE8M0: the scale is 2^127, the infinity the largest code
    (which stands for one again) and the rest as they are under that scale."""
    F = lib()
    n = 256
    h = inputs(2, n, 9)
    h[:, 0], h[:, 1], h[:, 2] = math.inf, 3e38, 1.0
    h[1, 0] = -math.inf
    q, scale = fill((2, n), torch.uint8), torch.ones(1, device="cuda")
    hq, hs = fill((2, n), torch.uint8), fill((2, 2), sdt(sfmt))
    F.fp8_act_checkpoint(h, None, F.ACT_SILU, q, scale=scale, keep_sfmt=sfmt, h_q=hq, h_scales=hs)
    check_kept(hq[:, 128:], hs[1:], h[:, 128:], sfmt)
    assert int(q[0, 0]) == 0x7E and int(q[1, 0]) & 0x7F == 0  # the activation's limits
    if sfmt:
        assert (hs[0] == 254).all()
        assert [int(c) for c in hq[:, 0]] == [0x7E, 0xFE]
        assert (hq[:, 1] == 0x3E).all()  # 1.75 x 2^127 of 3e38
        assert (hq[:, 2:128] & 0x7F == 0).all()
    else:
        assert torch.isinf(hs[0]).all()
        assert (hq[:, 0] & 0x7F == 0x7F).all() and (hq[:, 1:128] & 0x7F == 0).all()
    da, dh = torch.ones_like(h), fill((2, n), BF)
    ones, one = torch.full((2, n), 0x38, dtype=torch.uint8, device="cuda"), torch.ones((2, 2), device="cuda")
    us = one if sfmt == 0 else torch.full((2, 2), 127, dtype=torch.uint8, device="cuda")
    du = fill((2, n), BF)
    F.fp8_act_checkpoint_backward(da, F.ACT_SILU, hq, hs, ones, us, keep_sfmt=sfmt, dh=dh, du=du)
    assert dh[:, 128:].isfinite().all() and du[:, 128:].isfinite().all()
    if sfmt:
        assert dh[0, :2].tolist() == [1.0, 1.0] and (dh[:, 2:128] == 0.5).all()
        assert float(du[0, 0]) == math.inf and float(du[0, 1]) == float(torch.tensor(1.75 * 2.0 ** 127, dtype=BF))
        assert float(dh[1, 0]) == 0.0 and float(du[1, 0]) == 0.0
    else:
        assert dh[:, :128].isnan().all() and du[:, :128].isnan().all()


@SFMT
@pytest.mark.parametrize("fmt", [0, 1])
def test_a_group_with_a_nan(sfmt, fmt):
    """The rest of the group under a scale of 1, in codes and checkpoints."""
    F = lib()
    n = 256
    h = inputs(2, n, 10)
    h[0, 5], h[1, 200] = math.nan, math.nan
    q, sc = fill((2, n), torch.uint8), fill((2, 2), sdt(sfmt))
    hq, hs = fill((2, n), torch.uint8), fill((2, 2), sdt(sfmt))
    F.fp8_act_checkpoint(h, None, F.ACT_NONE, q, scales=sc, fmt=fmt, sfmt=sfmt, keep_sfmt=sfmt, h_q=hq,
                         h_scales=hs)
    one = 127 if sfmt else 1.0
    assert all(float(s[0, 0]) == one and float(s[1, 1]) == one for s in (sc, hs))
    for got, f8 in ((q, (torch.float8_e4m3fn, torch.float8_e5m2)[fmt]), (hq, torch.float8_e4m3fn)):
        v = got.view(f8).float()
        want = h.float().to(f8).float()
        for r, c in ((0, slice(0, 128)), (1, slice(128, 256))):
            assert torch.equal(torch.nan_to_num(v[r, c], 9e9), torch.nan_to_num(want[r, c], 9e9))
    check_kept(hq[:1, 128:], hs[1:, :1], h[:1, 128:], sfmt)
    dh = fill((2, n), BF)
    F.fp8_act_checkpoint_backward(torch.ones_like(h), F.ACT_SILU, hq, hs, keep_sfmt=sfmt, dh=dh)
    assert torch.equal(dh.isnan(), h.isnan())
