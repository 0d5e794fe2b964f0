"""Argument checks of the RMS norm and linear-epilogue calls (host only: the
checks run before any CUDA call, so a well-formed call answers "no device"
here)."""
import ctypes

import pytest
import torch

import fp8_quantized_gemm_gb300 as F

HAS_GPU = torch.cuda.is_available()
INVALID, MISALIGNED, UNSUPPORTED, NO_DEVICE = -1, -2, -3, -6
P = 1 << 20  # stands for an aligned device pointer


def call(name, *structs):
    return getattr(F._lib, name)(*[ctypes.addressof(s) for s in structs], None)


def norm(**kw):
    d = dict(x=P, residual=P, w=P, dt=0, w_dt=1, M=4, K=256, ld_x=256, ld_residual=256, eps=1e-5,
             mode=0, fmt=0, sfmt=0, scale=P, q=P, scales=None, sum_out=P, ld_sum=256, y_out=None,
             ld_y=0, inv_rms=P, amax_out=None)
    d.update(kw)
    return call("fp8_rmsnorm_quantize", F.RmsNorm(**d))


@pytest.mark.parametrize("kw,status", [
    (dict(x=None), INVALID), (dict(q=None), INVALID), (dict(M=-1), INVALID), (dict(K=0), INVALID),
    (dict(dt=2), INVALID), (dict(w_dt=5), INVALID), (dict(fmt=2), INVALID), (dict(mode=3), INVALID),
    (dict(eps=-1.0), INVALID), (dict(eps=float("nan")), INVALID), (dict(scale=None), INVALID),
    (dict(amax_out=P), INVALID),                       # amax over the scale
    (dict(mode=1, scales=None), INVALID), (dict(mode=1, scales=P, sfmt=7), INVALID),
    (dict(mode=1, scales=P, amax_out=P + 16), UNSUPPORTED),
    (dict(K=264, ld_x=264, ld_residual=264, ld_sum=264), MISALIGNED),
    (dict(mode=2, scales=P, K=144), MISALIGNED),       # MX words: K % 128
    (dict(K=16400, ld_x=16400, ld_residual=16400, ld_sum=16400), UNSUPPORTED),
    (dict(ld_x=255), INVALID), (dict(ld_residual=100), INVALID), (dict(ld_x=260), MISALIGNED),
    (dict(x=P + 8), MISALIGNED), (dict(sum_out=P + 2), MISALIGNED), (dict(q=P + 8), MISALIGNED),
    (dict(y_out=P, ld_y=128), INVALID), (dict(inv_rms=P + 2), MISALIGNED), (dict(w=P + 4), MISALIGNED)])
def test_norm(kw, status):
    assert norm(**kw) == status


def grad(**kw):
    d = dict(dy=P, r=P, w=P, d_residual=P, inv_rms=P, dy_dt=1, dt=0, w_dt=1, M=40, K=256, ld_dy=256,
             ld_r=256, ld_dres=256, ld_dx=256, dx=P, dw=P, accumulate_dw=0, q=P, fmt=1, scale=P,
             amax_out=P + 16, workspace=P, workspace_bytes=F.fp8_rmsnorm_backward_workspace(40, 256))
    d.update(kw)
    return call("fp8_rmsnorm_backward", F.RmsNormGrad(**d))


@pytest.mark.parametrize("kw,status", [
    (dict(dy=None), INVALID), (dict(r=None), INVALID), (dict(inv_rms=None), INVALID),
    (dict(dx=None), INVALID), (dict(dy_dt=3), INVALID), (dict(accumulate_dw=2), INVALID),
    (dict(scale=None), INVALID), (dict(amax_out=P), INVALID), (dict(fmt=4), INVALID),
    (dict(q=None), UNSUPPORTED),                       # an amax without codes
    (dict(workspace=None), INVALID), (dict(workspace_bytes=F.fp8_rmsnorm_backward_workspace(40, 256) - 1), INVALID),
    (dict(workspace=P + 8), MISALIGNED), (dict(K=250), MISALIGNED), (dict(K=32768), UNSUPPORTED),
    (dict(ld_dx=248), INVALID), (dict(ld_dy=257), MISALIGNED), (dict(dw=P + 1), MISALIGNED)])
def test_norm_grad(kw, status):
    assert grad(**kw) == status


def problem(**kw):
    d = dict(a=P, b=P, sa=P, sb=P, M=64, N=64, K=64, fa=0, fb=0, out_dt=1, accumulate=0, c=P, ldc=64,
             a_layout=0, b_layout=0, bias=P)
    d.update(kw)
    return F.GemmProblem(**d)


def epilogue(**kw):
    d = dict(act=3, residual=P, residual_dt=1, ld_residual=64, pre=P, ld_pre=64, q=P, q_fmt=0,
             q_scale=P, q_amax=P + 16)
    d.update(kw)
    return F.LinearEpilogue(**d)


PROBLEMS = [(dict(a=None), INVALID), (dict(M=0), INVALID), (dict(K=20), MISALIGNED),
            (dict(fa=2), INVALID), (dict(ldc=63), INVALID), (dict(accumulate=1, out_dt=0), UNSUPPORTED),
            (dict(c=P + 1), MISALIGNED), (dict(sa=None), INVALID),
            (dict(adamw=ctypes.pointer(F.AdamwEpilogue())), UNSUPPORTED)]
CODES = [(dict(act=6), INVALID), (dict(act=-1), INVALID), (dict(pre=P, ld_pre=63), INVALID),
         (dict(pre=P + 1), MISALIGNED), (dict(q_scale=None), INVALID), (dict(q_amax=P), INVALID),
         (dict(q_fmt=3), INVALID), (dict(q=None), UNSUPPORTED), (dict(q_scale=P + 2), MISALIGNED)]


@pytest.mark.parametrize("kw,status", PROBLEMS)
def test_tensor_problem(kw, status):
    assert call("fp8_gemm_tensor_epilogue", problem(**kw), epilogue()) == status


@pytest.mark.parametrize("kw,status", CODES + [
    (dict(ld_residual=10), INVALID), (dict(residual_dt=2), INVALID), (dict(residual=P + 1), MISALIGNED)])
def test_tensor_epilogue(kw, status):
    assert call("fp8_gemm_tensor_epilogue", problem(), epilogue(**kw)) == status


def test_output_may_be_missing_only_with_codes():
    rc = call("fp8_gemm_tensor_epilogue", problem(c=None, ldc=0), epilogue(q=None, q_amax=None))
    assert rc == INVALID
    if not HAS_GPU:
        assert call("fp8_gemm_tensor_epilogue", problem(c=None, ldc=0), epilogue()) == NO_DEVICE


def act_grad(p=None, **kw):
    d = dict(act=4, pre=P, ld_pre=64, q=P, q_fmt=1, q_scale=P, q_amax=P + 16, dbias=P,
             accumulate_dbias=0, workspace=P, workspace_bytes=F.fp8_act_backward_workspace(64, 64))
    d.update(kw)
    return call("fp8_gemm_tensor_act_backward", problem(**dict(bias=None, **(p or {}))),
                F.ActGradEpilogue(**d))


@pytest.mark.parametrize("kw,status", CODES + [
    (dict(pre=None), INVALID), (dict(workspace=None), INVALID), (dict(workspace_bytes=F.fp8_act_backward_workspace(64, 64) - 1), INVALID),
    (dict(workspace=P + 4), MISALIGNED), (dict(accumulate_dbias=3), INVALID), (dict(dbias=P + 2), MISALIGNED)])
def test_act_grad(kw, status):
    assert act_grad(**kw) == status


def test_act_grad_takes_no_bias():
    assert call("fp8_gemm_tensor_act_backward", problem(),
                F.ActGradEpilogue(act=4, pre=P, ld_pre=64)) == UNSUPPORTED


def group(ep=True, **kw):
    d = dict(a=P, sa=P, b=P, sb=P, sfmt=0, m=8, n=64, k=128, bias=None, c=P, ldc=64, e={})
    d.update(kw)
    e = epilogue(q=None, q_amax=None, **d.pop("e"))
    return F._lib.fp8_gemm_group_epilogue(
        d["a"], d["sa"], d["b"], d["sb"], d["sfmt"], d["m"], d["n"], d["k"], d["bias"],
        ctypes.addressof(e) if ep else None, d["c"], d["ldc"], None)


def test_group():
    assert group(ep=False) == INVALID
    assert group(c=None) == INVALID
    assert group(k=144) == MISALIGNED
    assert group(sfmt=2) == INVALID
    assert group(ldc=10) == INVALID
    assert group(e=dict(act=9)) == INVALID
    e = epilogue()
    assert F._lib.fp8_gemm_group_epilogue(P, P, P, P, 0, 8, 64, 128, None, ctypes.addressof(e), P, 64,
                                          None) == UNSUPPORTED  # no codes here
    if not HAS_GPU:
        assert group() == NO_DEVICE


def test_well_formed_calls_reach_the_device():
    if HAS_GPU:
        pytest.skip("stand-in pointers")
    assert norm() == NO_DEVICE and grad() == NO_DEVICE and act_grad() == NO_DEVICE
    assert norm(M=0, x=None, q=None) == NO_DEVICE
    assert call("fp8_gemm_tensor_epilogue", problem(), epilogue()) == NO_DEVICE


def test_workspace_sizes():
    """At least the partial sums, nothing for an empty or refused shape."""
    assert F.fp8_act_backward_workspace(33, 100) >= 2 * 100 * 4
    assert F.fp8_act_backward_workspace(0, 16) == 0
    assert F.fp8_rmsnorm_backward_workspace(3, 256) >= 3 * 256 * 4
    assert F.fp8_rmsnorm_backward_workspace(0, 256) == 0
    assert F.fp8_rmsnorm_backward_workspace(8, 100) == 0
    assert F.fp8_rmsnorm_backward_workspace(1 << 20, 4096) >= 152 * 4096 * 4


def test_python_checks():
    x = torch.zeros(4, 32)
    with pytest.raises(ValueError):
        F.fp8_rmsnorm_quantize(x, None, 1e-5, F.E4M3, x, scale=x, scales=x)
    with pytest.raises(ValueError):
        F.fp8_rmsnorm_quantize(x, None, 1e-5, F.E4M3, x)
    with pytest.raises(ValueError):
        F.fp8_rmsnorm_quantize(x, None, 1e-5, F.E4M3, x, scale=x)  # not on the GPU
    with pytest.raises(ValueError):
        F.fp8_rmsnorm_quantize(x, None, 1e-5, F.E4M3, x, scale=x, residual=torch.zeros(4, 16))
