"""Scales, biases and offsets that are no multiple of their element size are
refused before any device call (host only: stand-in pointers)."""
import ctypes

import pytest

import fp8_quantized_gemm_gb300 as F

MISALIGNED = -2
P, ODD = 1 << 20, (1 << 20) + 2  # stand for aligned and misaligned device pointers
L = F._lib


def problem(**kw):
    d = dict(a=P, b=P, sa=P, sb=P, M=64, N=64, K=64, fa=0, fb=0, out_dt=1, accumulate=0, c=P, ldc=64,
             a_layout=0, b_layout=0, bias=P)
    d.update(kw)
    return F.GemmProblem(**d)


@pytest.mark.parametrize("kw", [dict(sa=ODD), dict(sb=ODD), dict(bias=ODD), dict(bias=P + 1)])
def test_tensor_calls(kw):
    p, e = problem(**kw), F.LinearEpilogue(act=1)
    at = ctypes.addressof
    assert L.fp8_gemm_tensor_epilogue(at(p), at(e), None) == MISALIGNED
    assert L.fp8_gemm_tensor_grouped(ctypes.pointer(p), 1, None) == MISALIGNED
    if "bias" not in kw:
        g = F.ActGradEpilogue(act=1, pre=P, ld_pre=64)
        q = problem(**dict(kw, bias=None))
        assert L.fp8_gemm_tensor_act_backward(at(q), at(g), None) == MISALIGNED
        assert L.fp8_gemm_tensor(P, 0, P, 0, kw.get("sa", P), kw.get("sb", P), 64, 64, 64, 1, P, 64, 0,
                                 None) == MISALIGNED


@pytest.mark.parametrize("sa,sb,bias", [(ODD, P, P), (P, ODD, P), (P, P, ODD)])
@pytest.mark.parametrize("m", [8, 512])
def test_group_calls(sa, sb, bias, m):
    e = F.LinearEpilogue(act=1)
    assert L.fp8_gemm_group_epilogue(P, sa, P, sb, 0, m, 256, 128, bias, ctypes.addressof(e), P, 256,
                                     None) == MISALIGNED
    assert L.fp8_gemm_group_bias(P, sa, P, sb, 0, m, 256, 128, bias, P, 256, None) == MISALIGNED
    if bias == P:
        assert L.fp8_gemm_group(P, sa, P, sb, 0, m, 256, 128, P, 256, None) == MISALIGNED
        assert L.fp8_gemm_group_noalloc(P, sa, P, sb, 0, m, 256, 128, P, 256, None) == MISALIGNED
        assert L.fp8_gemm_group32(P, sa, P, sb, m, 256, 128, P, 256, None) == MISALIGNED
        assert L.fp8_gemm_group_experts(P, sa, P, sb, 0, P, 2, m, 256, 128, P, 256, None) == MISALIGNED


def test_byte_scales_need_no_alignment():
    if not F.torch.cuda.is_available():  # past the checks: no device here
        assert L.fp8_gemm_group(P, ODD + 1, P, ODD, 1, 512, 256, 128, P, 256, None) == -6


def test_expert_offsets_and_global_factors():
    assert L.fp8_gemm_group_experts(P, P, P, P, 1, ODD, 2, 512, 256, 128, P, 256, None) == MISALIGNED
    for f in (L.fp8_gemm_mx, L.fp8_gemm_mx_rows):
        assert f(P, P, ODD, P, P, P, 64, 64, 128, 1, P, 64, None) == MISALIGNED
        assert f(P, P, P, P, P, ODD, 64, 64, 128, 1, P, 64, None) == MISALIGNED
