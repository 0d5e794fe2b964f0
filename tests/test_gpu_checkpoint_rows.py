"""The checkpointed activation and its gradient: what a row's codes and scales are
depends on that row's group alone.  Every comparison here is of bytes: the same
rows in a call without and with other rows whose scales leave the common range
(tiny and huge values, infinities, NaN), and in a call of their own.
"""
import math

import pytest
import torch

from gpu_util import lib

pytestmark = pytest.mark.gpu

BF = torch.bfloat16
# rows that take a walk's first, last and middle tiles, alone and beside each other
AT = [0, 77, 78, 5000, 9003, 16384, 16388]
BY = [1e-32, 1e32, math.inf, math.nan, 1e-32, -math.inf, 1e32]


def randn(shape, seed, std=1.3):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda") * std).clamp(-7, 7).to(BF)


def sdt(sfmt):
    return torch.uint8 if sfmt else torch.float32


def forward(h, u, act, mode, fmt, sfmt, keep_sfmt):
    F = lib()
    m, n = h.shape
    g = (n + 127) // 128
    out = dict(q=torch.zeros((m, n), dtype=torch.uint8, device="cuda"))
    kw, kept = {}, {}
    if mode == "tensor":
        kw["scale"] = torch.full((1,), 0.05, device="cuda")
    else:
        out["scales"] = kw["scales"] = torch.zeros((g, m), dtype=sdt(sfmt), device="cuda")
    for name, x in (("h", h), ("u", u)):
        if x is not None:
            kept[name + "_q"] = torch.zeros((m, n), dtype=torch.uint8, device="cuda")
            kept[name + "_scales"] = torch.zeros((g, m), dtype=sdt(keep_sfmt), device="cuda")
    F.fp8_act_checkpoint(h, u, act, out["q"], fmt=fmt, sfmt=sfmt, keep_sfmt=keep_sfmt, **kw, **kept)
    return {**out, **kept}


def backward(da, kept, act, mode, fmt, sfmt, keep_sfmt, parts):
    F = lib()
    m, n = da.shape
    g = (n + 127) // 128
    out, kw = {}, {}
    for x in parts:
        out["d%s_q" % x] = torch.zeros((m, n), dtype=torch.uint8, device="cuda")
        if mode == "tensor":
            kw["scale_d" + x] = torch.full((1,), 1e-5, device="cuda")
        else:
            out["d%s_scales" % x] = torch.zeros((g, m), dtype=sdt(sfmt), device="cuda")
    F.fp8_act_checkpoint_backward(da, act, keep_sfmt=keep_sfmt, fmt=fmt, sfmt=sfmt, **kept, **out,
                                  **kw)
    return out


def same(a, b, rows, cols):
    """Codes of rows and columns (whole groups), and their scales, are the same bytes."""
    for key in a:
        x, y = a[key], b[key]
        if key.endswith("scales"):
            x, y = x[cols.start // 128:(cols.stop + 127) // 128, rows], y[cols.start // 128:(cols.stop + 127) // 128, rows]
        else:
            x, y = x[rows, cols], y[rows, cols]
        assert torch.equal(x.contiguous().view(torch.uint8), y.contiguous().view(torch.uint8)), key


@pytest.mark.parametrize("act,gate,mode,fmt,sfmt,keep_sfmt", [
    ("SILU", True, "group", 0, 0, 0), ("SILU", True, "group", 1, 1, 1), ("SILU", False, "group", 0, 0, 1),
    ("GELU_TANH", True, "tensor", 0, 0, 0), ("GELU_TANH", False, "group", 0, 1, 0),
    ("GELU", True, "group", 0, 0, 1), ("GELU", False, "tensor", 1, 0, 1), ("RELU2", False, "group", 0, 0, 0)])
def test_rows_beside_extreme_ones(act, gate, mode, fmt, sfmt, keep_sfmt):
    """Extreme values in the second group of a few rows: every other row, and these
    rows' other groups, are as without them (every CTA walks over several tiles)."""
    act = getattr(lib(), "ACT_" + act)
    m, n = 16389, 272
    h, u, da = randn((m, n), 1), randn((m, n), 2) if gate else None, randn((m, n), 3, 1e-3)
    at, by = torch.tensor(AT, device="cuda"), torch.tensor(BY, device="cuda")[:, None]
    other = torch.ones(m, dtype=torch.bool, device="cuda")
    other[at] = False
    every = torch.ones_like(other)
    parts = ("h", "u") if gate else ("h",)
    clean = forward(h, u, act, mode, fmt, sfmt, keep_sfmt)
    kept = {k: v for k, v in clean.items() if k[0] in "hu"}
    grads = backward(da, kept, act, mode, fmt, sfmt, keep_sfmt, parts)

    def check(a, b):
        same(a, b, other, slice(0, n))
        same(a, b, every, slice(0, 128))
        same(a, b, every, slice(256, n))

    hx = h.clone()
    hx[at, 128:256] = (hx[at, 128:256].float() * by).to(BF)
    check(forward(hx, u, act, mode, fmt, sfmt, keep_sfmt), clean)
    if gate:
        ux = u.clone()
        ux[at, 128:256] = (ux[at, 128:256].float() * by).to(BF)
        check(forward(h, ux, act, mode, fmt, sfmt, keep_sfmt), clean)
    dx = da.clone()
    dx[at, 128:256] = (dx[at, 128:256].float() * by).to(BF)
    check(backward(dx, kept, act, mode, fmt, sfmt, keep_sfmt, parts), grads)
    for name in parts:  # the checkpoints of extreme values
        kx = {k: v.clone() for k, v in kept.items()}
        if keep_sfmt:
            kx[name + "_scales"][1, at] = torch.tensor([3, 250, 254, 255, 1, 230, 170], dtype=torch.uint8, device="cuda")
        else:
            kx[name + "_scales"][1, at] *= by[:, 0].abs()
        check(backward(da, kx, act, mode, fmt, sfmt, keep_sfmt, parts), grads)


@pytest.mark.parametrize("gate,sfmt", [(True, 0), (False, 1)])
def test_a_batch_and_its_rows_alone(gate, sfmt):
    """Rows of common and of extreme size in one call, and each in a call of its own."""
    F = lib()
    m, n = 64, 400
    h, u = randn((m, n), 4), randn((m, n), 5) if gate else None
    scale = torch.tensor([1.0, 1e-32, 1e32, 1.0, math.inf, 1.0, math.nan, 1e-38], device="cuda")
    h = (h.float() * scale.repeat(m // 8)[:, None]).to(BF)
    da = (randn((m, n), 6).float() * scale.flip(0).repeat(m // 8)[:, None]).to(BF)
    parts = ("h", "u") if gate else ("h",)
    all_f = forward(h, u, F.ACT_SILU, "group", 0, sfmt, sfmt)
    kept = {k: v for k, v in all_f.items() if k[0] in "hu"}
    all_b = backward(da, kept, F.ACT_SILU, "group", 0, sfmt, sfmt, parts)
    for r in range(m):
        one = forward(h[r:r + 1], None if u is None else u[r:r + 1], F.ACT_SILU, "group", 0, sfmt, sfmt)
        one_kept = {k: v for k, v in one.items() if k[0] in "hu"}
        one.update(backward(da[r:r + 1], one_kept, F.ACT_SILU, "group", 0, sfmt, sfmt, parts))
        for key, t in {**all_f, **all_b}.items():
            t = t[:, r:r + 1] if key.endswith("scales") else t[r:r + 1]
            assert torch.equal(t.contiguous().view(torch.uint8), one[key].view(torch.uint8)), (r, key)


@pytest.mark.parametrize("gate,each", [(True, 256), (False, 256), (False, 1024)])
def test_long_walks(gate, each):
    """More tiles than resident CTAs take `each` of: the rows of a short pattern,
    repeated, with extreme ones at the walks' ends and between."""
    F = lib()
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    n, period = 128, 64
    times = (32 * (sms * (3 if gate else 4) * each + 5)) // period
    m = times * period
    small_h, small_u = randn((2 * period, n), 7), randn((2 * period, n), 8) if gate else None
    small_h[period:] = (small_h[period:].float() * 1e-32).to(BF)
    da = randn((2 * period, n), 9, 1e-3)
    parts = ("h", "u") if gate else ("h",)
    ref = forward(small_h, small_u, F.ACT_SILU, "group", 0, 0, 0)
    ref.update(backward(da, {k: v for k, v in ref.items() if k[0] in "hu"}, F.ACT_SILU, "group", 0, 0, 0, parts))
    which = torch.zeros(times, dtype=torch.int64, device="cuda")  # 1: a period of extreme rows
    which[[0, 1, times // 3, times // 2, times - 2, times - 1]] = 1
    rows = (which[:, None] * period + torch.arange(period, device="cuda")).view(-1)
    h, u = small_h[rows], small_u[rows] if gate else None
    out = forward(h, u, F.ACT_SILU, "group", 0, 0, 0)
    kept = {k: v for k, v in out.items() if k[0] in "hu"}
    del h, u
    out.update(backward(da[rows], kept, F.ACT_SILU, "group", 0, 0, 0, parts))
    for key, t in out.items():
        if key.endswith("scales"):
            assert torch.equal(t, ref[key][:, rows]), key
        else:
            assert torch.equal(t, ref[key][rows]), key
