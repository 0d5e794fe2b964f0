"""The mixture-of-experts layer stage by stage: every call that the layer makes is
recorded, and its result is compared with the definition on the operands that the
stage before has left (so that each bound is that of one call: the products' by the
oracle, the rest as in the calls' own tests)."""
import pytest
import torch

from gpu_util import lib
from oracle import gemm as OG
from oracle import quantize as OQ
from test_gpu_act_checkpoint import REL, check_group, check_kept, kept_values, slope, value
from test_gpu_experts import HALF, order

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


def randn(shape, seed, std):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(shape, generator=g, device="cuda") * std


def product(q, s, w, ws, offsets, sfmt, out, live):
    """out = the oracle's expert products of codes q and weights w."""
    m, k = q.shape
    name = "ue8m0" if sfmt else "f32"
    a = OG.dequant_operand(q.cpu().numpy()[:live], "e4m3",
                           OQ.expand(OQ.group_scale_values(s.t().cpu().numpy()[:live], name), live, k, 1, 128))
    n = w.shape[1]
    b = [OG.dequant_operand(w[e].cpu().numpy(), "e4m3",
                            OQ.expand(OQ.group_scale_values(ws[e].cpu().numpy(), name), n, k, 128, 128))
         for e in range(w.shape[0])]
    c, err = OG.gemm_experts(a, b, offsets.cpu().numpy())
    ok, worst = OG.check(out.float().cpu().numpy()[:live], c, err, "bf16")
    assert ok, worst


@pytest.mark.parametrize("t,s,e,d,ffn,drop,sfmt,keep_sfmt,res", [
    (150, 3, 6, 384, 256, 0.3, 0, 1, True), (400, 2, 8, 512, 384, 0.0, 1, 0, False),
    (1500, 2, 4, 256, 128, 0.2, 0, 0, True)])
def test_stages(monkeypatch, t, s, e, d, ffn, drop, sfmt, keep_sfmt, res):
    F = lib()
    from fp8_quantized_gemm_gb300.experts import ExpertsMLP
    mlp = ExpertsMLP(randn((e, 2 * ffn, d), 1, d ** -0.5).to(BF), randn((e, d, ffn), 2, ffn ** -0.5).to(BF),
                     sfmt=sfmt, backward=True, keep_sfmt=keep_sfmt)
    calls = []
    for name in ("fp8_experts_sort", "fp8_experts_gather", "fp8_gemm_group_experts", "fp8_act_checkpoint",
                 "fp8_experts_combine", "fp8_experts_combine_backward", "fp8_act_checkpoint_backward"):
        def call(*args, _fn=getattr(F, name), _name=name, **kw):
            calls.append((_name, args, kw))
            return _fn(*args, **kw)
        monkeypatch.setattr(F, name, call)
    x, w = randn((t, d), 3, 1.0).to(BF), torch.softmax(randn((t, s), 4, 1.0), 1)
    ids = torch.randint(0, e, (t, s), device="cuda", generator=torch.Generator("cuda").manual_seed(5))
    if drop:
        u = torch.rand((t, s), device="cuda", generator=torch.Generator("cuda").manual_seed(6))
        ids = torch.where(u < drop, -1, ids)
    r = randn((t, d), 7, 1.0).to(BF) if res else None
    out = mlp(x, ids, w, residual=r, keep=True)
    dout = randn((t, d), 8, 1e-2).to(BF)
    dx, dw = mlp.backward(dout)
    torch.cuda.synchronize()
    assert [c[0][4:] for c in calls] == [
        "experts_sort", "experts_gather", "gemm_group_experts", "act_checkpoint", "gemm_group_experts",
        "experts_combine", "experts_combine_backward", "gemm_group_experts", "act_checkpoint_backward",
        "gemm_group_experts", "experts_combine"]
    # rows
    offsets, rows = calls[0][1][2], calls[0][1][3]
    want = order(ids, e)
    assert torch.equal(offsets, want[0]) and torch.equal(rows, want[1])
    live = int(offsets[-1])
    pair = torch.nonzero(rows.reshape(-1) >= 0).squeeze(1)
    at, tok = rows.reshape(-1)[pair].long(), pair // s
    # codes of x
    xq, xs = calls[1][2]["q"], calls[1][2]["scales"]
    lq, ls = torch.empty((t, d), dtype=torch.uint8, device="cuda"), torch.empty((d // 128, t), dtype=xs.dtype, device="cuda")
    F.fp8_quantize_token_group(x, F.E4M3, sfmt, lq, ls)
    assert torch.equal(xq[at], lq[tok]) and torch.equal(xs[:, at], ls[:, tok])
    # h | u
    hu = calls[2][1][6]
    product(xq, xs, *mlp.w13, offsets, sfmt, hu, live)
    h, u = hu[:live, :ffn], hu[:live, ffn:]
    # a, and the checkpoints
    aq, kw = calls[3][1][3], calls[3][2]
    a = value(h.double(), "silu") * u.double()
    check_group(aq[:live], kw["scales"][:, :live], a, REL * a.abs() + 1e-38, 0, sfmt)
    vals = {}
    for name, v in (("h", h), ("u", u)):
        q, sc = kw[name + "_q"][:live], kw[name + "_scales"][:, :live]
        check_kept(q, sc, v, keep_sfmt)
        vals[name] = kept_values(q, sc, keep_sfmt)
    # y, out
    y = calls[4][1][6]
    product(aq, kw["scales"], *mlp.w2, offsets, sfmt, y, live)
    terms = torch.zeros((t * s, d), dtype=torch.float64, device="cuda")
    terms[pair] = y.double()[at] * w.double().reshape(-1)[pair][:, None]
    terms = terms.view(t, s, d)
    sums, mag = terms.sum(1), terms.abs().sum(1)
    if res:
        sums, mag = sums + r.double(), mag + r.double().abs()
    tol = (s + 1) * 2.0 ** -24 * mag * (1 + 2.0 ** -7)
    assert ((out.double() - sums).abs() <= tol + HALF[BF] * (sums.abs() + tol) + 1e-40).all()
    # codes of w dout, dw
    kw = calls[6][2]
    v = dout.double()[tok] * w.double().reshape(-1)[pair][:, None]
    back = torch.empty((live, d), dtype=torch.float64, device="cuda")
    back[at] = v
    check_group(kw["q"][:live], kw["scales"][:, :live], back, 2.0 ** -23 * back.abs(), 0, sfmt)
    prod = torch.zeros((t * s, d), dtype=torch.float64, device="cuda")
    prod[pair] = dout.double()[tok] * y.double()[at]
    assert ((dw.double().view(-1) - prod.sum(1)).abs() <= 80 * 2.0 ** -24 * prod.abs().sum(1) + 1e-40).all()
    # da, dh | du
    da = calls[7][1][6]
    product(kw["q"], kw["scales"], *mlp.w2t, offsets, sfmt, da, live)
    g, kw = da[:live].double(), calls[8][2]
    sl = slope(vals["h"], "silu")
    dh, du = g * sl * vals["u"], g * value(vals["h"], "silu")
    err = REL * g.abs() * sl.abs().clamp_min(1.0) * vals["u"].abs() + 1e-38
    check_group(kw["dh_q"][:live].contiguous(), kw["dh_scales"][:, :live], dh, err, 0, sfmt)
    check_group(kw["du_q"][:live].contiguous(), kw["du_scales"][:, :live], du, REL * du.abs() + 1e-38, 0, sfmt)
    # the next product's operand is dh | du
    gq, gs = calls[9][1][0], calls[9][1][1]
    assert torch.equal(gq[:live, :ffn], kw["dh_q"][:live]) and torch.equal(gq[:live, ffn:], kw["du_q"][:live])
    assert torch.equal(gs[:, :live], torch.cat([kw["dh_scales"], kw["du_scales"]])[:, :live])
    rows_dx = calls[9][1][6]
    product(gq, gs, *mlp.w13t, offsets, sfmt, rows_dx, live)
    terms = torch.zeros((t * s, d), dtype=torch.float64, device="cuda")
    terms[pair] = rows_dx.double()[at]
    terms = terms.view(t, s, d)
    sums, mag = terms.sum(1), terms.abs().sum(1)
    tol = (s + 1) * 2.0 ** -24 * mag * (1 + 2.0 ** -7)
    assert ((dx.double() - sums).abs() <= tol + HALF[BF] * (sums.abs() + tol) + 1e-40).all()
    assert F.fp8_get_last_device_error() == (0, 0)
