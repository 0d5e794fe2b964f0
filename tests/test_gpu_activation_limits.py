"""Activations and their slopes at infinite arguments: the limits of the
definitions, exactly (0, 1, the argument itself; relu2's slope is infinite).
Finite values near the top of fp32 reach the slopes as infinities too, through
the bf16 pre-activation."""
import math

import pytest
import torch

from gpu_util import lib

pytestmark = pytest.mark.gpu

INF = math.inf
ACTS = ["none", "relu", "relu2", "silu", "gelu_tanh", "gelu"]
LEFT = {"none": -INF}                        # act(-inf), 0 elsewhere
SLOPES = {"none": (1, 1), "relu2": (0, INF)}  # at -inf and +inf, (0, 1) elsewhere
# the general kernel on one tile, split K in a cluster, CTA pairs
SHAPES = [(5, 48, 32), (33, 520, 2064), (2048, 2560, 160)]


def zeros(*s):
    return torch.zeros(s, dtype=torch.uint8, device="cuda")


def bias_of(n):
    b = torch.ones(n, device="cuda")
    b[::4], b[1::4], b[3] = INF, -INF, math.nan
    return b


@pytest.mark.parametrize("m,n,k", SHAPES)
@pytest.mark.parametrize("name", ACTS)
def test_values(m, n, k, name):
    F = lib()
    one, b = torch.ones(1, device="cuda"), bias_of(n)
    out, pre = torch.empty((m, n), device="cuda"), torch.empty((m, n), device="cuda").bfloat16()
    q, amax = zeros(m, n), torch.empty(1, device="cuda")
    F.fp8_gemm_tensor_epilogue(zeros(m, k), 0, zeros(n, k), 0, one, one, out, bias=b,
                               act=ACTS.index(name), pre_out=pre, q=q, q_scale=one, q_amax=amax)
    left = LEFT.get(name, 0.0)
    assert (out[:, ::4] == INF).all() and (out[:, 1::4] == left).all()
    assert torch.isnan(out[:, 3]).all() and torch.isfinite(out[:, 2::4]).all()
    assert (pre[:, ::4] == INF).all() and (pre[:, 1::4] == -INF).all()
    v = q.view(torch.float8_e4m3fn).float()
    assert (v[:, ::4] == 448).all() and (v[:, 1::4] == max(left, -448)).all()
    assert torch.isnan(v[:, 3]).all() and math.isnan(amax.item())


@pytest.mark.parametrize("m,sfmt", [(3, 0), (70, 1), (300, 1), (300, 0)])
@pytest.mark.parametrize("name", ACTS)
def test_group_values(m, sfmt, name):
    F = lib()
    n, k, st = 256, 256, (torch.float32, torch.uint8)[sfmt]
    unit = 127 if sfmt else 1
    sa = torch.full((k // 128, m), unit, dtype=st, device="cuda")
    sb = torch.full((n // 128, k // 128), unit, dtype=st, device="cuda")
    out = torch.empty((m, n), dtype=torch.bfloat16, device="cuda")
    F.fp8_gemm_group_epilogue(zeros(m, k), sa, zeros(n, k), sb, sfmt, out, bias=bias_of(n),
                              act=ACTS.index(name))
    assert (out[:, ::4] == INF).all() and (out[:, 1::4] == LEFT.get(name, 0.0)).all()
    assert torch.isnan(out[:, 3]).all() and torch.isfinite(out[:, 2::4]).all()


@pytest.mark.parametrize("m,n,k", SHAPES)
@pytest.mark.parametrize("name", ACTS)
def test_slopes(m, n, k, name):
    """A gradient of exactly one in every place: K codes of 1, scale 1 / K."""
    F = lib()
    ones = torch.ones(1).to(torch.float8_e4m3fn).view(torch.uint8).item()
    a, b = (torch.full(s, ones, dtype=torch.uint8, device="cuda") for s in ((m, k), (n, k)))
    kk = 1 << (k - 1).bit_length()  # a power of two: the product K / kk is exact
    sa, sb = torch.full((1,), 1.0 / kk, device="cuda"), torch.ones(1, device="cuda")
    top = torch.finfo(torch.float32).max  # rounds to infinity in bf16
    pre = torch.ones((m, n), device="cuda")
    pre[:, ::4], pre[:, 1::4], pre[:, 3], pre[:, 7] = INF, -INF, math.nan, top
    pre = pre.bfloat16()
    assert (pre[:, 7] == INF).all()
    out, db = torch.empty((m, n), device="cuda"), torch.empty(n, device="cuda")
    F.fp8_gemm_tensor_act_backward(a, 0, b, 0, sa, sb, pre, ACTS.index(name), out=out, dbias=db)
    lo, hi = SLOPES.get(name, (0, 1))
    g = k / kk
    assert (out[:, ::4] == g * hi).all() and (out[:, 7] == g * hi).all()
    assert (out[:, 1::4] == g * lo).all()
    assert torch.isfinite(out[:, 2::4]).all() and (name == "none" or torch.isnan(out[:, 3]).all())
    assert not torch.isnan(db[::4]).any() and not torch.isnan(db[1::4]).any()
