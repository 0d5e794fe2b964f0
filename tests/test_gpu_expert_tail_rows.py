"""fp8_gemm_group_experts on operands with more rows than the experts own
(offsets[E] < M, as fp8_experts_sort leaves them where pairs are dropped): the
experts' rows against the oracle, the rows behind them left as they were although
the operand's codes and scales there are NaN.  On CTA pairs, one CTA (FP32
scales), the UE8M0 kernel and the block-scaled one on E8M0 words."""
import pytest
import torch

from gpu_util import lib
from oracle import gemm as OG
from test_gpu_gemm import expert_operands

pytestmark = pytest.mark.gpu

# counts, N, K, rows behind the last expert's
CASES = [([5, 0, 17], 256, 256, 100),                    # at most 256 rows
         ([130, 0, 257, 3], 384, 384, 61),               # the tail begins inside a tile
         ([128, 256], 256, 256, 300),                    # on a tile's border, 1.2 tiles of it
         ([700, 0, 1, 1100, 255, 257], 1024, 384, 999)]  # enough tiles for CTA pairs


@pytest.mark.parametrize("sfmt", ["f32", "ue8m0"])
@pytest.mark.parametrize("counts,n,k,tail", CASES)
def test_rows_behind_the_experts(sfmt, counts, n, k, tail):
    F = lib()
    qa, sa, qb, sb, offs, c, e, m = expert_operands(len(counts), sum(counts), n, k, sfmt,
                                                    seed=n + tail, counts=counts)
    q = torch.full((m + tail, k), 0x7F, dtype=torch.uint8, device="cuda")
    q[:m] = qa
    if sfmt == "f32":
        s = torch.full((k // 128, m + tail), float("nan"), device="cuda")
    else:
        s = torch.full((k // 128, m + tail), 255, dtype=torch.uint8, device="cuda")
    s[:, :m] = sa
    code = F.SCALE_F32 if sfmt == "f32" else F.SCALE_UE8M0
    try:
        for pairs in (1, 0):
            F.fp8_set_option(F.OPT_GEMM_CTA_PAIRS, pairs)
            out = torch.full((m + tail, n), -7.0, dtype=torch.bfloat16, device="cuda")
            F.fp8_gemm_group_experts(q, s, qb, sb, code, offs, out)
            torch.cuda.synchronize()
            ok, worst = OG.check(out[:m].float().cpu().numpy(), c, e, "bf16")
            assert ok, (pairs, worst)
            assert (out[m:] == -7.0).all(), pairs
            # no expert owns a row
            out.fill_(-7.0)
            F.fp8_gemm_group_experts(q, s, qb, sb, code, torch.zeros_like(offs), out)
            assert (out == -7.0).all(), pairs
    finally:
        F.fp8_set_option(F.OPT_GEMM_CTA_PAIRS, 1)
    assert F.fp8_get_last_device_error()[0] == 0
