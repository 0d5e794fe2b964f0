"""gather where a warp takes two windows of 512 columns at once (short lists of many
tokens), and on both sides of that rule: the quantizer's bytes, rows as they are, and
codes moved."""
import pytest
import torch

from gpu_util import lib
from test_gpu_experts import DT, choices, filled, group_codes, order, pitched, randn

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("t,s,k,dt,sfmt,fmt,drop,pad", [
    (8200, 2, 1024, "bf16", 0, 0, 0.1, 8), (5200, 1, 1552, "bf16", 1, 1, 0.0, 0),
    (3000, 4, 3600, "f32", 0, 0, 0.2, 8), (8300, 3, 528, "f32", 1, 0, 0.0, 0),
    (2300, 2, 3584, "bf16", 0, 1, 0.3, 16),   # seven windows
    (9000, 1, 1040, "bf16", 0, 0, 0.0, 0),    # three: one at a time, but codes moved
    (7400, 2, 1024, "f32", 1, 1, 0.1, 0)])    # not enough of them for codes that are formed
def test_gather(t, s, k, dt, sfmt, fmt, drop, pad):
    F = lib()
    _, rows, _ = order(choices(t, s, 8, t + k, drop), 8)
    m, g, st = t * s + 5, (k + 127) // 128, torch.uint8 if sfmt else torch.float32
    x = randn((t, k), DT[dt], 1, 2.0)
    x[:, ::97] *= 30
    x[0, :k // 2] = 0
    x[7, 3], x[t - 1, k - 1], x[t // 2, k // 2] = float("nan"), 3e38, 1e-37
    pair = torch.nonzero(rows.reshape(-1) >= 0).squeeze(1)
    at, tok = rows.reshape(-1)[pair].long(), pair // s
    tq, ts = group_codes(x, sfmt, fmt)
    nan = x.isnan()  # (its group is compared with the library's own quantizer alone)
    wq, wsc, wout = filled((m, k), torch.uint8), filled((g, m), st), filled((m, k), DT[dt])
    wq[at], wout[at] = tq[tok], x[tok]
    wsc[:, at] = ts[:, tok]
    skip = torch.zeros((m, g), dtype=torch.bool, device="cuda")
    skip[at, 0] = tok == 7
    cols = skip.repeat_interleave(128, 1)[:, :k]

    def check(q, sc):
        assert torch.equal(q[~cols], wq[~cols]) and torch.equal(sc[~skip.t()], wsc[~skip.t()])

    q, sc, out = filled((m, k), torch.uint8), filled((g, m), st), filled((m, k), DT[dt])
    F.fp8_experts_gather(pitched(x, pad), rows, q=q, scales=sc, fmt=fmt, sfmt=sfmt, out=out)
    check(q, sc)
    assert torch.equal(out.view(torch.uint8), wout.view(torch.uint8))
    lq, ls = torch.empty((t, k), dtype=torch.uint8, device="cuda"), torch.empty((g, t), dtype=st, device="cuda")
    F.fp8_quantize_token_group(x, fmt, sfmt, lq, ls)
    got, want = q[at, :128], lq[tok, :128]  # with the NaN's group
    is_nan = nan[tok, :128]
    assert torch.equal(got[~is_nan], want[~is_nan]) and torch.equal(sc[0, at], ls[0, tok])
    q2, sc2 = filled((m, k), torch.uint8), filled((g, m), st)
    F.fp8_experts_gather(lq, rows, q=q2, scales=sc2, fmt=fmt, sfmt=sfmt, x_scales=ls)
    assert torch.equal(q2[at], lq[tok]) and torch.equal(sc2[:, at], ls[:, tok])
    check(q2, sc2)
    out2 = filled((m, k), DT[dt])
    F.fp8_experts_gather(pitched(x, pad), rows, out=out2)
    assert torch.equal(out2.view(torch.uint8), wout.view(torch.uint8))
