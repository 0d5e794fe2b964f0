"""The activation checkpointed in 8 bits, against the definitions in 64 bits
(plain torch, none of the library's code).

Tolerances.  The activations run on the hardware base-2 exponential and
reciprocal: with |z| <= 7 the exponent's argument (at most 40, from fp32
products) is off by 40 x 3 x 2^-24, the two instructions by 2^-22 each, gelu's
tail polynomial by 1.6e-7 = 2^-22.5: below 2^-16 of the value for each factor of
a product.  REL = 2^-16.  A slope is a difference of terms of magnitude at most
1.2 (2 |z| for relu2), so its error is taken relative to max(1, |slope|).  A
code is then off by half a step of the format plus that error over its scale,
and the scale itself, formed from such values, by REL and three roundings.
"""
import math

import pytest
import torch

from gpu_util import lib

pytestmark = pytest.mark.gpu

REL = 2.0 ** -16
F8 = (torch.float8_e4m3fn, torch.float8_e5m2)
TOP = (448.0, 57344.0)
MANT, EMIN = (3, 2), (-6, -14)
BF = torch.bfloat16
ACTS = ["none", "relu", "relu2", "silu", "gelu_tanh", "gelu"]


def value(z, act):
    if act == "relu":
        return z.clamp_min(0)
    if act == "relu2":
        return z.clamp_min(0) ** 2
    if act == "silu":
        return z * torch.sigmoid(z)
    if act == "gelu_tanh":
        return 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)))
    if act == "gelu":
        return 0.5 * z * torch.special.erfc(-z / math.sqrt(2))
    return z


def slope(z, act):
    if act == "none":
        return torch.ones_like(z)
    if act == "relu":  # (0 at 0)
        return (z > 0).to(z.dtype)
    z = z.clone().requires_grad_(True)
    return torch.autograd.grad(value(z, act).sum(), z)[0]


def half_step(v, fmt):
    e = torch.floor(torch.log2(v.abs().clamp_min(2.0 ** EMIN[fmt])))
    return torch.exp2(e - MANT[fmt] - 1)


def pow2(b):
    return torch.exp2(b.double() - 127)


def groups(v):
    m, n = v.shape
    g = (n + 127) // 128
    return torch.nn.functional.pad(v, (0, g * 128 - n)).view(m, g, 128)


def check_group(q, s, want, err, fmt, sfmt):
    """Group codes q [M, N] and stored scales s [G, M] of want (64 bits), whose
    fp32 form may be off by err."""
    m, n = want.shape
    top, slack = groups(want.abs()).amax(2), groups(err).amax(2)
    got = pow2(s.t()) if sfmt else s.t().double()
    ideal = torch.where(top > 0, top / TOP[fmt], torch.ones_like(top))
    room = slack / TOP[fmt] + 2.0 ** -22 * ideal
    if sfmt:
        ok = (got >= ideal - room) & (got / 2 < ideal + room)
    else:
        ok = (got - ideal).abs() <= room
    # a group within its error of zero may have become all zeros (scale 1)
    ok |= (top <= slack) & (got == 1.0)
    assert ok.all()
    u = (groups(want) / got[:, :, None]).flatten(1)[:, :n].clamp(-TOP[fmt], TOP[fmt])
    tol = (groups(err) / got[:, :, None]).flatten(1)[:, :n] + 2.0 ** -22 * u.abs()
    bad = (q.view(F8[fmt]).double() - u).abs() > half_step(u, fmt) * (1 + 1e-6) + 2 * tol
    assert not bad.any(), int(bad.sum())


def check_tensor(q, amax, scale, want, err, fmt):
    s = float(scale)
    u = (want / s).clamp(-TOP[fmt], TOP[fmt])
    bad = (q.view(F8[fmt]).double() - u).abs() > half_step(u, fmt) * (1 + 1e-6) + 2 * err / s + 2.0 ** -22 * u.abs()
    assert not bad.any(), int(bad.sum())
    top = want.abs().max()
    assert abs(float(amax.double() - top)) <= float(err.max()) + 2.0 ** -23 * float(top)


def quantizer(x, sfmt):
    """The bytes a checkpoint must hold: fp8_quantize_token_group's, in torch."""
    xg = groups(x.float())
    top = xg.abs().amax(2)
    # (not top / 448.0: torch multiplies by the rounded reciprocal of a scalar)
    s = torch.where(top > 0, top / torch.full_like(top, 448.0), torch.ones_like(top))
    if sfmt:
        man, e = torch.frexp(s)
        e = torch.where(man == 0.5, e - 1, e)
        s, kept = torch.ldexp(torch.ones_like(s), e), (e + 127).to(torch.uint8)
    else:
        kept = s
    q = (xg / s[:, :, None]).clamp(-448, 448).to(F8[0]).flatten(1)[:, :x.shape[1]]
    return q.contiguous().view(torch.uint8), kept.t().contiguous()


def check_kept(q, s, x, sfmt):
    """A checkpoint of bf16 x: the quantizer's scales, and codes of x times the
    scale's reciprocal (2^-23 off) rounded once more: 2^-22 and half a step."""
    _, ws = quantizer(x, sfmt)
    assert torch.equal(s, ws)
    sv = (pow2(ws) if sfmt else ws.double()).t()[:, :, None]
    u = (groups(x.double()) / sv).flatten(1)[:, :x.shape[1]]
    bad = (q.view(F8[0]).double() - u).abs() > half_step(u, 0) * (1 + 1e-6) + 2.0 ** -22 * u.abs()
    assert not bad.any(), int(bad.sum())


def kept_values(q, s, sfmt):
    """The values that a checkpoint stands for, in 64 bits."""
    s = pow2(s) if sfmt else s.double()
    return (groups(q.view(F8[0]).double()) * s.t()[:, :, None]).flatten(1)[:, :q.shape[1]]


def inputs(m, n, seed, std=1.3):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn((m, n), generator=g, device="cuda") * std).clamp(-7, 7).to(BF)


def fill(shape, dt):
    return torch.full(shape, 0xA5 if dt == torch.uint8 else -7.0, dtype=dt, device="cuda")


def sdt(sfmt):
    return torch.uint8 if sfmt else torch.float32


CASES = [  # m, n, act, gate, mode, fmt, sfmt, keep_sfmt, valid, wide
    (1, 16, "silu", True, "group", 0, 0, 0, None, False),
    (1, 2048, "silu", True, "group", 0, 1, 1, None, True),
    (33, 144, "gelu", True, "tensor", 0, 0, 1, None, False),
    (31, 128, "gelu_tanh", False, "group", 0, 0, 0, 17, False),
    (64, 528, "relu2", True, "group", 1, 0, 0, 64, True),
    (257, 1040, "silu", True, "tensor", 1, 0, 0, 100, True),
    (130, 272, "none", True, "group", 0, 0, 1, 0, False),
    (100, 640, "relu", False, "tensor", 0, 0, 0, 99, False),
    (2, 14336, "gelu", False, "group", 1, 1, 0, None, False),
    (1000, 2064, "gelu_tanh", True, "tensor", 0, 0, 0, None, True)]


def arguments(m, n, wide, gate, seed):
    if wide:  # halves of one product
        hu = inputs(m, 2 * n, seed)
        return hu[:, :n], hu[:, n:] if gate else None
    return inputs(m, n, seed), inputs(m, n, seed + 1) if gate else None


@pytest.mark.parametrize("m,n,act,gate,mode,fmt,sfmt,keep_sfmt,valid,wide", CASES)
def test_forward(m, n, act, gate, mode, fmt, sfmt, keep_sfmt, valid, wide):
    F = lib()
    h, u = arguments(m, n, wide, gate, m + n)
    h[0, :n // 2] = 0
    live = m if valid is None else valid
    h[live:] = float("nan")  # rows that hold nothing are not read
    g = (n + 127) // 128
    vr = None if valid is None else torch.tensor([valid], dtype=torch.int32, device="cuda")
    q, out = fill((m, n), torch.uint8), fill((m, n), BF)
    kw, scale, amax, sc = {}, None, None, None
    if mode == "tensor":
        scale = torch.full((1,), 30.0 / TOP[fmt], device="cuda")
        amax = torch.full((1,), 9e9, device="cuda")
        kw = dict(scale=scale, amax_out=amax)
    else:
        sc = fill((g, m), sdt(sfmt))
        kw = dict(scales=sc, sfmt=sfmt)
    names = ("h", "u") if gate else ("h",)
    kept = {}
    for name in names:
        kept[name + "_q"], kept[name + "_scales"] = fill((m, n), torch.uint8), fill((g, m), sdt(keep_sfmt))

    def run(**more):
        F.fp8_act_checkpoint(h, u, ACTS.index(act), q, fmt=fmt, valid_rows=vr, **kw, **more)

    run(out=out, keep_sfmt=keep_sfmt, **kept)
    hd, ud = h[:live].double(), u[:live].double() if gate else None
    want = value(hd, act) * ud if gate else value(hd, act)
    err = REL * want.abs() + 1e-38
    if mode == "tensor":
        if live:
            check_tensor(q[:live], amax, scale, want, err, fmt)
        else:
            assert float(amax) == 0.0
    elif live:
        check_group(q[:live], sc[:, :live], want, err, fmt, sfmt)
    assert ((out[:live].double() - want).abs() <= 2.0 ** -8 * want.abs() * (1 + REL) + err).all()
    for name, x in zip(names, (h, u)):
        check_kept(kept[name + "_q"][:live], kept[name + "_scales"][:, :live], x[:live], keep_sfmt)
    # rows behind the valid ones are as they were
    for t in [q, out] + [kept[x + "_q"] for x in names]:
        assert (t[live:] == (0xA5 if t.dtype == torch.uint8 else -7.0)).all()
    for t in ([sc] if sc is not None else []) + [kept[x + "_scales"] for x in names]:
        assert (t[:, live:] == (0xA5 if t.dtype == torch.uint8 else -7.0)).all()
    # without checkpoints and the bf16 copy: the same codes
    q0, a0 = q.clone(), None if amax is None else amax.clone()
    q.fill_(0xA5)
    run()
    assert torch.equal(q, q0) and (amax is None or torch.equal(amax, a0))


@pytest.mark.parametrize("m,n,act,gate,mode,fmt,sfmt,keep_sfmt,valid,wide", CASES)
def test_backward(m, n, act, gate, mode, fmt, sfmt, keep_sfmt, valid, wide):
    F = lib()
    h, u = arguments(m, n, wide, gate, m + n)
    g, live = (n + 127) // 128, m if valid is None else valid
    vr = None if valid is None else torch.tensor([valid], dtype=torch.int32, device="cuda")
    da = inputs(m, n, 77, 1e-3)
    da[live:] = float("nan")
    names = ("h", "u") if gate else ("h",)
    kept, vals = {}, {}
    for name, x in zip(names, (h, u)):
        kept[name + "_q"], kept[name + "_scales"] = quantizer(x, keep_sfmt)
        vals[name] = kept_values(kept[name + "_q"], kept[name + "_scales"], keep_sfmt)[:live]
    both = fill((m, 2 * n), torch.uint8) if wide else None
    outs, kw = {}, {}
    for i, name in enumerate(names):
        outs["d" + name + "_q"] = both[:, i * n:(i + 1) * n] if wide else fill((m, n), torch.uint8)
        outs["d" + name] = fill((m, n), BF)
        if mode == "tensor":
            kw["scale_d" + name] = torch.full((1,), 2e-2 / TOP[fmt] * (i + 1), device="cuda")
            kw["amax_d" + name] = torch.full((1,), 9e9, device="cuda")
        else:
            kw["d" + name + "_scales"] = fill((g, m), sdt(sfmt))
    F.fp8_act_checkpoint_backward(da, ACTS.index(act), keep_sfmt=keep_sfmt, fmt=fmt, sfmt=sfmt,
                                  valid_rows=vr, **kept, **outs, **kw)
    d, hv = da[:live].double(), vals["h"]
    sl = slope(hv, act)
    want = {"dh": d * sl}
    err = {"dh": REL * d.abs() * sl.abs().clamp_min(1.0)}
    if gate:
        want = {"dh": want["dh"] * vals["u"], "du": d * value(hv, act)}
        err = {"dh": err["dh"] * vals["u"].abs(), "du": REL * want["du"].abs()}
    for name in want:
        w, e = want[name], err[name] + 1e-38
        got = outs[name][:live].double()
        assert ((got - w).abs() <= 2.0 ** -8 * w.abs() + 2 * e).all()
        if mode == "group" and live:
            check_group(outs[name + "_q"][:live], kw[name + "_scales"][:, :live], w, e, fmt, sfmt)
        elif live:
            check_tensor(outs[name + "_q"][:live], kw["amax_" + name], kw["scale_" + name], w, e, fmt)
        elif mode == "tensor":
            assert float(kw["amax_" + name]) == 0.0
        assert (outs[name + "_q"][live:] == 0xA5).all() and (outs[name][live:] == -7.0).all()
    # codes alone, rows alone: the same
    for part in ("_q", ""):
        again = {}
        for name in names:
            again["d" + name + part] = torch.full_like(outs["d" + name + part], 0 if part else -1)
        more = kw if part else {}
        F.fp8_act_checkpoint_backward(da, ACTS.index(act), keep_sfmt=keep_sfmt, fmt=fmt, sfmt=sfmt,
                                      valid_rows=vr, **kept, **again, **more)
        for key, t in again.items():
            assert torch.equal(t[:live], outs[key][:live])


@pytest.mark.parametrize("act", ["silu", "gelu_tanh", "gelu"])
def test_backward_against_differences(act):
    """dh and du against central differences of act(h) u in 64 bits at the kept
    values: a step of 1e-4 leaves 1e-8 of the third derivative (below 1)."""
    F = lib()
    m, n = 8, 256
    (hq, hs), (uq, us) = quantizer(inputs(m, n, 1), 0), quantizer(inputs(m, n, 2), 0)
    hv, uv = kept_values(hq, hs, 0), kept_values(uq, us, 0)
    da = torch.ones((m, n), dtype=BF, device="cuda")
    dh, du = torch.empty_like(da), torch.empty_like(da)
    F.fp8_act_checkpoint_backward(da, ACTS.index(act), hq, hs, uq, us, dh=dh, du=du)
    eps = 1e-4
    want = (value(hv + eps, act) - value(hv - eps, act)) / (2 * eps) * uv
    assert ((dh.double() - want).abs() <= 2.0 ** -8 * want.abs() + 2 * REL * (1 + uv.abs())).all()
    want = value(hv, act)
    assert ((du.double() - want).abs() <= 2.0 ** -8 * want.abs() + 2 * REL).all()


def test_limits_and_non_finite_arguments():
    """Infinite arguments take the activation's limits; a checkpoint keeps a NaN
    as one, and a group with an infinity as NaN (fp32 scales)."""
    F = lib()
    n = 256
    h = inputs(4, n, 3)
    h[0, 0], h[1, 0], h[2, 0] = float("inf"), -float("inf"), float("nan")
    scale = torch.full((1,), 0.05, device="cuda")
    for act in ("relu", "silu", "gelu_tanh", "gelu"):
        q, out = fill((4, n), torch.uint8), fill((4, n), BF)
        hq, hs = fill((4, n), torch.uint8), fill((2, 4), torch.float32)
        F.fp8_act_checkpoint(h, None, ACTS.index(act), q, scale=scale, out=out, h_q=hq, h_scales=hs)
        assert float(out[0, 0]) == float("inf") and float(out[1, 0]) == 0.0
        assert int(q[0, 0]) == 0x7E and int(q[1, 0]) & 0x7F == 0 and int(q[2, 0]) & 0x7F == 0x7F
        check_kept(hq[3:], hs[:, 3:], h[3:], 0)
        dh = fill((4, n), BF)
        F.fp8_act_checkpoint_backward(torch.ones_like(h), ACTS.index(act), hq, hs, dh=dh)
        nan = torch.isnan(dh)
        assert nan[0, :128].all() and nan[1, :128].all() and nan[2, 0]
        assert not nan[:, 128:].any() and not nan[2, 1:].any() and not nan[3].any()


def test_extreme_scales():
    """Values whose group scales leave the range of the rounded reciprocal."""
    F = lib()
    n = 128
    h = (inputs(3, n, 4) * torch.tensor([[1e-36], [1.0], [1e36]], device="cuda")).to(BF)
    q, sc = fill((3, n), torch.uint8), fill((1, 3), torch.float32)
    hq, hs = fill((3, n), torch.uint8), fill((1, 3), torch.float32)
    F.fp8_act_checkpoint(h, None, F.ACT_NONE, q, scales=sc, h_q=hq, h_scales=hs)
    check_kept(hq, hs, h, 0)
    check_group(q, sc, h.double(), torch.zeros_like(h.double()), 0, 0)


@pytest.mark.parametrize("act,gate,fmt", [("silu", True, 0), ("gelu", False, 1)])
def test_extreme_rows_among_many(act, gate, fmt):
    """Rows whose scales leave the common range among rows that stay, where every
    CTA walks over several tiles."""
    F = lib()
    m, n = 16389, 272
    at = torch.tensor([0, 77, 5000, 9001, 16384, 16388], device="cuda")
    by = torch.tensor([1e-32, 1e32, 1e32, 1e-32, 1e-32, 1e32], device="cuda")[:, None]
    h, u = inputs(m, n, 21), inputs(m, n, 22) if gate else None
    da, g = inputs(m, n, 23, 1e-3), 3
    h[at] = (h[at].float() * by).to(BF)
    da[at + 1 - 2 * (at == m - 1).long()] *= 1e-32

    def run():
        r = dict(q=fill((m, n), torch.uint8), scales=fill((g, m), torch.float32))
        kept = {}
        for x in ("h", "u") if gate else ("h",):
            kept[x + "_q"], kept[x + "_scales"] = fill((m, n), torch.uint8), fill((g, m), torch.float32)
            r["d%s_q" % x] = fill((m, n), torch.uint8)
            r["d%s_scales" % x] = fill((g, m), torch.float32)
        F.fp8_act_checkpoint(h, u, ACTS.index(act), r["q"], scales=r["scales"], fmt=fmt, **kept)
        F.fp8_act_checkpoint_backward(da, ACTS.index(act), fmt=fmt, **kept,
                                      **{k: v for k, v in r.items() if k[0] == "d"})
        return {**r, **kept}

    got = run()
    hv, dv = kept_values(got["h_q"], got["h_scales"], 0), da.double()
    check_kept(got["h_q"], got["h_scales"], h, 0)
    y = value(h.double(), act) * (u.double() if gate else 1.0)
    check_group(got["q"], got["scales"], y, REL * y.abs() + 1e-38, fmt, 0)
    sl = slope(hv, act)
    dh, err = dv * sl, REL * dv.abs() * sl.abs().clamp_min(1.0)
    if gate:
        uv = kept_values(got["u_q"], got["u_scales"], 0)
        check_kept(got["u_q"], got["u_scales"], u, 0)
        dh, err = dh * uv, err * uv.abs()
        du = dv * value(hv, act)
        check_group(got["du_q"], got["du_scales"], du, REL * du.abs() + 1e-38, fmt, 0)
    check_group(got["dh_q"], got["dh_scales"], dh, err + 1e-38, fmt, 0)


@pytest.mark.parametrize("act,gate,fmt", [("silu", True, 0), ("relu2", False, 1)])
def test_extreme_tensor_scales(act, gate, fmt):
    """Per-tensor scales beyond the range of the rounded reciprocal."""
    F = lib()
    m, n = 1000, 272
    h, u = inputs(m, n, 31), inputs(m, n, 32) if gate else None
    q, amax = fill((m, n), torch.uint8), fill((1,), torch.float32)
    kept, outs, kw, vals = {}, {}, {}, {}
    for name, x in zip(("h", "u"), (h, u)):
        if x is None:
            continue
        kept[name + "_q"], kept[name + "_scales"] = quantizer(x, 0)
        vals[name] = kept_values(kept[name + "_q"], kept[name + "_scales"], 0)
        outs["d%s_q" % name] = fill((m, n), torch.uint8)
        kw["scale_d" + name] = torch.full((1,), 2e-31 / TOP[fmt], device="cuda")
        kw["amax_d" + name] = fill((1,), torch.float32)
    da = inputs(m, n, 33, 1e-3) * 1e-29
    F.fp8_act_checkpoint_backward(da, ACTS.index(act), fmt=fmt, **kept, **outs, **kw)
    dv, sl = da.double(), slope(vals["h"], act)
    dh, err = dv * sl, REL * dv.abs() * sl.abs().clamp_min(1.0)
    if gate:
        dh, err = dh * vals["u"], err * vals["u"].abs()
        du = dv * value(vals["h"], act)
        check_tensor(outs["du_q"], kw["amax_du"], kw["scale_du"], du, REL * du.abs(), fmt)
    check_tensor(outs["dh_q"], kw["amax_dh"], kw["scale_dh"], dh, err, fmt)
    if gate:  # forward: the gate's rows carry the size
        w = (u.float() * 1e-32).to(BF)
        scale = torch.full((1,), 5e-32 / TOP[fmt], device="cuda")
        F.fp8_act_checkpoint(h, w, ACTS.index(act), q, scale=scale, amax_out=amax, fmt=fmt)
        y = value(h.double(), act) * w.double()
        check_tensor(q, amax, scale, y, REL * y.abs(), fmt)


def test_rows_beyond_32_bit_offsets():
    F = lib()
    m, n, first = 300016, 14400, 300000  # 4.3e9 elements
    vals = inputs(16, n, 5)
    h = torch.zeros((m, n), dtype=BF, device="cuda")
    h[first:] = vals
    q, hq = (torch.zeros((m, n), dtype=torch.uint8, device="cuda") for _ in range(2))
    g = (n + 127) // 128
    sc, hs = torch.zeros((g, m), device="cuda"), torch.zeros((g, m), device="cuda")
    F.fp8_act_checkpoint(h, None, F.ACT_SILU, q, scales=sc, h_q=hq, h_scales=hs)
    wq, ws = hq[first:], hs[:, first:]
    check_kept(wq, ws, vals, 0)
    want = value(vals.double(), "silu")
    check_group(q[first:], sc[:, first:], want, REL * want.abs() + 1e-38, 0, 0)
    F.fp8_act_checkpoint_backward(h, F.ACT_SILU, hq, hs, dh_q=q, dh_scales=sc, fmt=F.E4M3)
    w = vals.double() * slope(kept_values(wq, ws, 0), "silu")
    check_group(q[first:], sc[:, first:], w, REL * vals.double().abs() + 1e-38, 0, 0)


def test_graph_replay_and_streams():
    """Captured and replayed on new inputs beside a direct call on another
    stream; the maxima are cleared by every replay."""
    F = lib()
    m, n = 100, 1040

    def buffers():
        d = dict(q=fill((m, n), torch.uint8), amax=fill((1,), torch.float32))
        for x in ("h", "u"):
            d[x + "_q"], d[x + "_scales"] = fill((m, n), torch.uint8), fill((9, m), torch.float32)
            d["d" + x], d["amax_" + x] = fill((m, n), torch.uint8), fill((1,), torch.float32)
        return d

    s1 = torch.full((1,), 0.05, device="cuda")
    s2 = torch.full((1,), 0.002, device="cuda")

    def run(h, u, da, b):
        kept = {k: b[k] for k in ("h_q", "h_scales", "u_q", "u_scales")}
        F.fp8_act_checkpoint(h, u, F.ACT_SILU, b["q"], scale=s1, amax_out=b["amax"], **kept)
        F.fp8_act_checkpoint_backward(da, F.ACT_SILU, dh_q=b["dh"], du_q=b["du"], scale_dh=s2,
                                      scale_du=s2, amax_dh=b["amax_h"], amax_du=b["amax_u"], **kept)

    sets = [(inputs(m, n, 3 * i, 2.0 - 0.5 * i), inputs(m, n, 3 * i + 1), inputs(m, n, 3 * i + 2, 0.1))
            for i in range(2)]
    want = []
    for x in sets:
        want.append(buffers())
        run(*x, want[-1])
    live, b = [t.clone() for t in sets[0]], buffers()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        run(*live, b)
    side, direct = torch.cuda.Stream(), buffers()
    torch.cuda.synchronize()
    for i in (0, 1):
        for t, src in zip(live, sets[i]):
            t.copy_(src)
        torch.cuda.synchronize()
        g.replay()
        with torch.cuda.stream(side):
            run(*sets[1 - i], direct)
        torch.cuda.synchronize()
        for key in b:
            assert torch.equal(b[key], want[i][key]) and torch.equal(direct[key], want[1 - i][key]), key


def test_trainer_with_8_bit_checkpoints():
    """SwiGLUTrainer(checkpoint="fp8"): the checkpoints are the codes of the h
    and u that the two products give, the codes of a, dh and du those of the
    formulas, and a captured step repeats a direct one."""
    F = lib()
    from fp8_quantized_gemm_gb300.mlp import A2, G1, G3, K1, K3, X1, SwiGLUTrainer
    T, d, ffn = 272, 256, 528
    w1, w3 = inputs(ffn, d, 1, 0.08), inputs(ffn, d, 2, 0.08)
    w2 = inputs(d, ffn, 3, 0.05)
    x, dy = inputs(T, d, 4), inputs(T, d, 5, 1e-2)
    tr = SwiGLUTrainer(w1, w3, w2, T, history=4, checkpoint="fp8")
    assert tr.h is None and tr.u is None
    for _ in range(3):  # the histories have seen data
        tr.step(x, dy)
    tr.forward_backward(x, dy)
    h, u = (torch.empty((T, ffn), dtype=BF, device="cuda") for _ in range(2))
    P = F.gemm_problem
    F.fp8_gemm_tensor_grouped([
        P(tr.xq, F.E4M3, w, F.E4M3, tr.scale[X1:X1 + 1], tr.scale[slot:slot + 1], y)
        for w, slot, y in ((tr.w1q, K1, h), (tr.w3q, K3, u))])
    vals = {}
    for name, y in (("h", h), ("u", u)):
        q, s = tr.kept[name + "_q"], tr.kept[name + "_scales"]
        check_kept(q, s, y, 0)
        vals[name] = kept_values(q, s, 0)
    want = value(h.double(), "silu") * u.double()
    check_tensor(tr.aq, tr.amax[A2:A2 + 1], tr.scale[A2], want, REL * want.abs() + 1e-30, 0)
    d_ = tr.da.double()
    sl = slope(vals["h"], "silu")
    for slot, q, w, e in (
            (G1, tr.dhq, d_ * sl * vals["u"], d_.abs() * sl.abs().clamp_min(1) * vals["u"].abs()),
            (G3, tr.duq, d_ * value(vals["h"], "silu"), (d_ * value(vals["h"], "silu")).abs())):
        check_tensor(q, tr.amax[slot:slot + 1], tr.scale[slot], w, REL * e + 1e-30, 1)
    a, b = (SwiGLUTrainer(w1, w3, w2, T, history=4, checkpoint="fp8") for _ in range(2))
    for t in (a, b):
        t.step(x, dy)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        a.step(x, dy)
    for _ in range(2):
        g.replay()
        b.step(x, dy)
    torch.cuda.synchronize()
    assert torch.equal(a.aq, b.aq) and torch.equal(a.dhq, b.dhq) and torch.equal(a.scale, b.scale)
    for p, q in zip(a.w_master, b.w_master):
        assert torch.equal(p, q)


def test_binding_refuses():
    F = lib()
    h = inputs(4, 256, 1)
    q = torch.empty((4, 256), dtype=torch.uint8, device="cuda")
    sc, one = torch.empty((2, 4), device="cuda"), torch.ones(1, device="cuda")
    with pytest.raises(ValueError):
        F.fp8_act_checkpoint(h, None, F.ACT_SILU, q)
    with pytest.raises(ValueError):
        F.fp8_act_checkpoint(h, None, F.ACT_SILU, q, scale=one, scales=sc)
    with pytest.raises(ValueError):
        F.fp8_act_checkpoint(h, h.float(), F.ACT_SILU, q, scale=one)
    with pytest.raises(ValueError):
        F.fp8_act_checkpoint(h, h[:2], F.ACT_SILU, q, scale=one)
    with pytest.raises(ValueError):
        F.fp8_act_checkpoint(h, None, F.ACT_SILU, q, scale=one, h_q=q)
    with pytest.raises(ValueError):
        F.fp8_act_checkpoint(h, None, F.ACT_SILU, q[:2], scale=one)
    with pytest.raises(ValueError):
        F.fp8_act_checkpoint(h.cpu(), None, F.ACT_SILU, q, scale=one)
    with pytest.raises(F.Fp8Error):
        F.fp8_act_checkpoint(h, h, F.ACT_SILU, q, scale=one, h_q=q.clone(), h_scales=sc)
    with pytest.raises(F.Fp8Error):
        F.fp8_act_checkpoint_backward(h, F.ACT_SILU, q, sc)
    with pytest.raises(ValueError):
        F.fp8_act_checkpoint_backward(h, F.ACT_SILU, q, sc, dh_q=q.clone(), dh_scales=sc,
                                      scale_dh=one)
    wide = torch.empty((4, 512), dtype=torch.uint8, device="cuda")
    with pytest.raises(ValueError):  # two pitches
        F.fp8_act_checkpoint_backward(h, F.ACT_SILU, q, sc, q, sc, dh_q=q.clone(), du_q=wide[:, :256],
                                      scale_dh=one, scale_du=one)
