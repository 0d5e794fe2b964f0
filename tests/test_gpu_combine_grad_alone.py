"""The gradient of combine where a warp takes a token alone: many tokens (7000: the
rule asks for 36 to 42 an SM) of one or two choices, rows of more than 512 columns.

Tolerances as in test_gpu_experts.py; dw: a lane adds four pairs per 256 columns,
112 fused steps at 7168 columns, then two halves and five shuffles: 120 steps of
2^-24 on the sum of the magnitudes.
"""
import math

import pytest
import torch

from gpu_util import lib
from test_gpu_experts import (DT, F8, FILL, REL, TOP, choices, filled, half_step, order, pitched,
                              randn)

pytestmark = pytest.mark.gpu

T, STEPS = 7000, 120

CASES = [  # s, k, x, dy, sfmt, fmt, weights, drop, pad
    (1, 7168, "bf16", "bf16", 0, 0, True, 0.1, 0), (2, 7168, "bf16", "bf16", 1, 0, True, 0.2, 8),
    (2, 4096, "bf16", "f32", 0, 1, True, 0.1, 0), (1, 1040, "bf16", "f32", 1, 1, False, 0.3, 16),
    (2, 1296, "f32", "bf16", 1, 0, True, 0.2, 0), (1, 7168, "f32", "bf16", 0, 0, True, 0.0, 8),
    (2, 2064, "f32", "f32", 1, 1, True, 0.1, 0), (1, 528, "f32", "f32", 0, 0, False, 0.5, 0)]


@pytest.mark.parametrize("s,k,dt,dydt,sfmt,fmt,weights,drop,pad", CASES)
def test_codes_rows_and_weights(s, k, dt, dydt, sfmt, fmt, weights, drop, pad):
    F = lib()
    _, rows, _ = order(choices(T, s, 16, k + s, drop), 16)
    m, g = T * s + 3, (k + 127) // 128
    dy = randn((T, k), DT[dydt], 1, 1e-3)
    dy[5, :k // 2] = 0
    x = randn((m, k), DT[dt], 2)
    w = randn((T, s), torch.float32, 3, 0.5) if weights else None
    q, sc = filled((m, k), torch.uint8), filled((g, m), torch.uint8 if sfmt else torch.float32)
    dx, dw = filled((m, k + pad), torch.float32), filled((T, s), torch.float32)
    F.fp8_experts_combine_backward(pitched(dy, pad), rows, w, x=pitched(x, pad), d_weights=dw, q=q,
                                   scales=sc, fmt=fmt, sfmt=sfmt, dx=dx[:, :k])
    pair = torch.nonzero(rows.reshape(-1) >= 0).squeeze(1)
    at, tok = rows.reshape(-1)[pair].long(), pair // s
    v = dy.double()[tok]
    want, mag = (torch.zeros(T * s, dtype=torch.float64, device="cuda") for _ in range(2))
    prod = v * x.double()[at]
    want[pair], mag[pair] = prod.sum(1), prod.abs().sum(1)
    del prod
    assert ((dw.double().view(-1) - want).abs() <= STEPS * 2.0 ** -24 * mag + 1e-40).all()
    if weights:
        v = v * w.reshape(-1)[pair].double()[:, None]
    assert ((dx[at, :k].double() - v).abs() <= 2.0 ** -24 * v.abs() + 1e-44).all()
    vp = torch.nn.functional.pad(v, (0, g * 128 - k)).view(-1, g, 128)
    top, got = vp.abs().amax(2), sc[:, at].t()
    scale = torch.where(top > 0, top / TOP[fmt], torch.ones_like(top))
    if sfmt:
        ge = torch.exp2(got.double() - 127)
        ok = (ge >= scale * (1 - REL)) & (ge / 2 < scale * (1 + REL))
        assert (ok | ((top == 0) & (got == 127))).all()
    else:
        ge = got.double()
        assert ((ge - scale).abs() <= REL * scale).all()
    u = (vp / ge[:, :, None]).view(-1, g * 128)[:, :k].clamp(-TOP[fmt], TOP[fmt])
    err = (q[at].view(F8[fmt]).double() - u).abs()
    assert (err <= half_step(u, fmt) * (1 + 1e-6) + REL * u.abs()).all()
    other = torch.ones(m, dtype=torch.bool, device="cuda")
    other[at] = False
    assert (q[other] == FILL).all() and (dx[other] == -7.0).all() and (dx[:, k:] == -7.0).all()
    assert (sc[:, other] == (FILL if sfmt else -7.0)).all()


@pytest.mark.parametrize("dt,dydt", [("bf16", "bf16"), ("f32", "bf16"), ("bf16", "f32")])
def test_dropped_pairs_beside_non_finite_gradients(dt, dydt):
    F = lib()
    s, k = 2, 1040
    _, rows, _ = order(choices(T, s, 4, 9, 0.4), 4)
    x, dy = randn((T * s, k), DT[dt], 1), randn((T, k), DT[dydt], 2)
    bad = torch.tensor([0, 1, 2, 3500, T - 1], device="cuda")
    dy[0, 3], dy[1, 300], dy[2, k - 1], dy[3500], dy[T - 1, 700] = math.inf, -math.inf, math.nan, math.inf, math.nan
    dw = filled((T, s), torch.float32)
    F.fp8_experts_combine_backward(dy, rows, torch.ones((T, s), device="cuda"), x=x, d_weights=dw)
    gone = rows < 0
    assert (dw[gone] == 0).all()
    assert gone[bad].any() and not dw[bad][~gone[bad]].isfinite().any()
    fine = ~gone
    fine[bad] = False
    prod = dy.double()[:, None] * x.double()[rows.clamp_min(0).long()]
    assert ((dw.double() - prod.sum(2)).abs() <= STEPS * 2.0 ** -24 * prod.abs().sum(2))[fine].all()


def test_a_token_alone_and_among_many():
    """The bytes of the codes do not depend on how many tokens the call holds."""
    F = lib()
    s, k, few = 2, 2064, 700  # (700: a CTA takes a token)
    dy, w = randn((T, k), torch.bfloat16, 4, 1e-3), randn((T, s), torch.float32, 5)
    rows = torch.arange(T * s, dtype=torch.int32, device="cuda").view(T, s)
    out = []
    for t in (T, few):
        q, sc = filled((t * s, k), torch.uint8), filled(((k + 127) // 128, t * s), torch.float32)
        F.fp8_experts_combine_backward(dy[:t], rows[:t].contiguous(), w[:t].contiguous(), q=q, scales=sc)
        out.append((q, sc))
    assert torch.equal(out[0][0][:few * s], out[1][0]) and torch.equal(out[0][1][:, :few * s], out[1][1])
