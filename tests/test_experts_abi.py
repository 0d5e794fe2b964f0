"""Argument checks of the expert-row and activation-checkpoint calls (host only:
the checks run before any CUDA call, so a well-formed call answers "no device"
here), and the rules their sources keep."""
import ctypes
import os
import re

import pytest
import torch

import fp8_quantized_gemm_gb300 as F

HAS_GPU = torch.cuda.is_available()
INVALID, MISALIGNED, UNSUPPORTED, NO_DEVICE = -1, -2, -3, -6
P = 1 << 20  # stands for an aligned device pointer
CSRC = os.path.join(os.path.dirname(F.__file__), "csrc")


def call(name, s):
    return getattr(F._lib, name)(ctypes.addressof(s), None)


def sort(**kw):
    d = dict(ids=P, id_dt=1, T=4, S=2, experts=8, offsets=2 * P, rows=3 * P, pairs=4 * P)
    d.update(kw)
    return F._lib.fp8_experts_sort(*d.values(), None)


@pytest.mark.parametrize("kw,status", [
    (dict(ids=None), INVALID), (dict(rows=None), INVALID), (dict(offsets=None), INVALID),
    (dict(id_dt=2), INVALID), (dict(T=-1), INVALID), (dict(S=0), INVALID),
    (dict(T=1 << 30, S=2), INVALID), (dict(experts=0), INVALID), (dict(experts=257), INVALID),
    (dict(ids=P + 4), MISALIGNED), (dict(id_dt=0, ids=P + 2), MISALIGNED),
    (dict(rows=P + 2), MISALIGNED), (dict(pairs=P + 1), MISALIGNED),
    (dict(offsets=P + 2), MISALIGNED), (dict(rows=P), INVALID), (dict(pairs=3 * P), INVALID)])
def test_sort(kw, status):
    assert sort(**kw) == status


def gather(**kw):
    d = dict(x=P, dt=0, ld_x=256, xq=None, x_scales=None, rows=P, T=4, S=2, K=256, M=8, fmt=0,
             sfmt=0, q=P, scales=P, out=P, ld_out=256)
    d.update(kw)
    return call("fp8_experts_gather", F.ExpertsGather(**d))


CODES = dict(x=None, out=None, xq=P, x_scales=P)


@pytest.mark.parametrize("kw,status", [
    (dict(x=None), INVALID), (dict(rows=None), INVALID), (dict(T=-1), INVALID),
    (dict(S=0), INVALID), (dict(M=-1), INVALID), (dict(K=0), INVALID), (dict(T=1 << 31), INVALID),
    (dict(dt=2), INVALID), (dict(fmt=2), INVALID), (dict(sfmt=2), INVALID),
    (dict(q=None), INVALID), (dict(scales=None), INVALID),
    (dict(q=None, scales=None, out=None), INVALID), (dict(K=264, ld_x=264, ld_out=264), MISALIGNED),
    (dict(ld_x=248), INVALID), (dict(ld_out=257), MISALIGNED), (dict(x=P + 8), MISALIGNED),
    (dict(q=P + 4), MISALIGNED), (dict(scales=P + 2), MISALIGNED), (dict(rows=P + 2), MISALIGNED),
    (dict(CODES, x=P), UNSUPPORTED), (dict(CODES, out=P), UNSUPPORTED),
    (dict(CODES, x_scales=None), INVALID), (dict(CODES, q=None, scales=None), INVALID),
    (dict(CODES, xq=P + 8), MISALIGNED), (dict(CODES, x_scales=P + 1), MISALIGNED)])
def test_gather(kw, status):
    assert gather(**kw) == status


def combine(**kw):
    d = dict(x=P, x_dt=0, ld_x=256, rows=P, weights=P, T=4, S=2, K=256, M=8, residual=P,
             ld_residual=256, out=2 * P, out_dt=0, ld_out=256)
    d.update(kw)
    return call("fp8_experts_combine", F.ExpertsCombine(**d))


@pytest.mark.parametrize("kw,status", [
    (dict(x=None), INVALID), (dict(out=None), INVALID), (dict(rows=None), INVALID),
    (dict(x_dt=2), INVALID), (dict(out_dt=-1), INVALID), (dict(K=8, ld_x=8), MISALIGNED),
    (dict(ld_x=8), INVALID), (dict(ld_residual=260), MISALIGNED), (dict(out=P + 2), MISALIGNED),
    (dict(residual=2 * P, ld_residual=512), INVALID),  # in place, another pitch
    (dict(weights=P + 2), MISALIGNED), (dict(ld_x=1 << 30), UNSUPPORTED)])
def test_combine(kw, status):
    assert combine(**kw) == status


def combine_grad(**kw):
    d = dict(dy=P, dy_dt=0, ld_dy=256, x=P, x_dt=0, ld_x=256, rows=P, weights=P, T=4, S=2, K=256,
             M=8, d_weights=P, q=P, scales=P, fmt=0, sfmt=0, dx=P, dx_dt=0, ld_dx=256)
    d.update(kw)
    return call("fp8_experts_combine_backward", F.ExpertsCombineGrad(**d))


@pytest.mark.parametrize("kw,status", [
    (dict(dy=None), INVALID), (dict(x=None), INVALID), (dict(rows=None), INVALID),
    (dict(dy_dt=2), INVALID), (dict(x_dt=2), INVALID), (dict(dx_dt=2), INVALID),
    (dict(fmt=3), INVALID), (dict(sfmt=3), INVALID), (dict(scales=None), INVALID),
    (dict(q=None), INVALID), (dict(q=None, scales=None, dx=None, d_weights=None), INVALID),
    (dict(K=120, ld_dy=120), MISALIGNED), (dict(ld_dy=128), INVALID), (dict(ld_x=255), INVALID),
    (dict(ld_dx=300), MISALIGNED), (dict(d_weights=P + 2), MISALIGNED), (dict(q=P + 8), MISALIGNED)])
def test_combine_grad(kw, status):
    assert combine_grad(**kw) == status


def act(**kw):
    d = dict(act=3, h=P, ld_h=512, u=P, ld_u=512, M=4, N=256, valid_rows=P, mode=1, fmt=0, sfmt=0,
             q=P, scale=None, scales=P, amax_out=None, keep_sfmt=0, h_q=P, h_scales=P, u_q=P,
             u_scales=P, out=P, ld_out=256)
    d.update(kw)
    return call("fp8_act_checkpoint", F.ActCheckpoint(**d))


TENSOR = dict(mode=0, scale=P, scales=None, amax_out=P + 16)


@pytest.mark.parametrize("kw,status", [
    (dict(h=None), INVALID), (dict(q=None), INVALID), (dict(M=-1), INVALID), (dict(N=0), INVALID),
    (dict(act=6), INVALID), (dict(act=-1), INVALID), (dict(fmt=2), INVALID), (dict(mode=3), INVALID),
    (dict(mode=2), UNSUPPORTED), (dict(sfmt=2), INVALID), (dict(keep_sfmt=2), INVALID),
    (dict(scales=None), INVALID), (dict(scale=P), INVALID), (dict(amax_out=P), UNSUPPORTED),
    (dict(TENSOR, scale=None), INVALID), (dict(TENSOR, amax_out=P), INVALID),
    (dict(TENSOR, scales=P), INVALID),
    (dict(h_q=None), INVALID), (dict(h_scales=None), INVALID), (dict(u_q=None), INVALID),
    (dict(u_q=None, u_scales=None), INVALID),  # a gate kept on one side only
    (dict(u=None), INVALID), (dict(h_q=None, h_scales=None), INVALID),
    (dict(N=200, ld_out=200), MISALIGNED), (dict(ld_h=248), INVALID), (dict(ld_u=257), MISALIGNED),
    (dict(h=P + 8), MISALIGNED), (dict(q=P + 8), MISALIGNED), (dict(h_q=P + 1), MISALIGNED),
    (dict(h_scales=P + 2), MISALIGNED), (dict(valid_rows=P + 2), MISALIGNED),
    (dict(ld_out=8), INVALID)])
def test_act(kw, status):
    assert act(**kw) == status


def act_grad(**kw):
    d = dict(act=3, da=P, ld_da=256, h_q=P, h_scales=P, u_q=P, u_scales=P, keep_sfmt=0, M=4, N=256,
             valid_rows=None, mode=1, fmt=0, sfmt=0, dh_q=P, du_q=P + 256, ld_q=512, scale_dh=None,
             scale_du=None, dh_scales=P, du_scales=P, amax_dh=None, amax_du=None, dh=P, du=P,
             ld_d=256)
    d.update(kw)
    return call("fp8_act_checkpoint_backward", F.ActCheckpointGrad(**d))


GTENSOR = dict(mode=0, scale_dh=P, scale_du=P + 16, amax_dh=P + 32, amax_du=P + 48)


@pytest.mark.parametrize("kw,status", [
    (dict(da=None), INVALID), (dict(h_q=None), INVALID), (dict(h_scales=None), INVALID),
    (dict(u_q=None), INVALID), (dict(u_scales=None), INVALID),
    (dict(u_q=None, u_scales=None), INVALID),  # du without a gate
    (dict(dh_q=None, du_q=None, dh=None, du=None), INVALID), (dict(act=9), INVALID),
    (dict(mode=2), UNSUPPORTED), (dict(mode=7), INVALID), (dict(dh_scales=None), INVALID),
    (dict(du_scales=None), INVALID), (dict(amax_dh=P), UNSUPPORTED), (dict(keep_sfmt=5), INVALID),
    (dict(sfmt=5), INVALID), (dict(fmt=2), INVALID), (dict(GTENSOR, scale_du=None), INVALID),
    (dict(GTENSOR, amax_dh=P), INVALID), (dict(GTENSOR, amax_du=P + 32), INVALID),
    (dict(GTENSOR, dh_q=None), UNSUPPORTED),  # a maximum without codes
    (dict(ld_q=240), INVALID), (dict(ld_q=520), MISALIGNED), (dict(du_q=P + 8), MISALIGNED),
    (dict(ld_d=100), INVALID), (dict(ld_da=260), MISALIGNED),
    (dict(N=264, ld_da=264, ld_d=264), MISALIGNED), (dict(h_scales=P + 1), MISALIGNED)])
def test_act_grad(kw, status):
    assert act_grad(**kw) == status


@pytest.mark.skipif(HAS_GPU, reason="would launch on stand-in pointers")
@pytest.mark.parametrize("fn,kw", [
    (sort, {}), (sort, dict(pairs=None)), (sort, dict(T=0, ids=None, rows=None)), (gather, {}),
    (gather, CODES), (gather, dict(q=None, scales=None)), (gather, dict(out=None)),
    (gather, dict(T=0, x=None, rows=None)), (combine, {}),
    (combine, dict(weights=None, residual=None)), (combine, dict(residual=2 * P)),
    (combine, dict(M=0, x=None)), (combine_grad, {}), (combine_grad, dict(weights=None, dx=None)),
    (combine_grad, dict(d_weights=None, x=None)), (act, {}), (act, TENSOR),
    (act, dict(u=None, u_q=None, u_scales=None)),
    (act, dict(h_q=None, h_scales=None, u_q=None, u_scales=None)), (act_grad, {}),
    (act_grad, GTENSOR), (act_grad, dict(dh=None, du=None)),
    (act_grad, dict(dh_q=None, du_q=None, dh_scales=None, du_scales=None)),
    (act_grad, dict(u_q=None, u_scales=None, du_q=None, du=None, du_scales=None)),
    (act, dict(M=0, h=None, u=None, q=None, scales=None, h_q=None, h_scales=None, u_q=None,
               u_scales=None))])
def test_well_formed_calls_reach_the_device_check(fn, kw):
    assert fn(**kw) == NO_DEVICE


@pytest.mark.parametrize("name", ["fp8_experts_gather", "fp8_experts_combine",
                                  "fp8_experts_combine_backward", "fp8_act_checkpoint",
                                  "fp8_act_checkpoint_backward"])
def test_null_descriptor(name):
    assert getattr(F._lib, name)(None, None) == INVALID


def test_programmatically_launched_sources_have_no_read_only_loads():
    """Every file that launches with programmatic stream serialization through
    launch.h, and the headers whose loads those kernels use."""
    def source(name):
        with open(os.path.join(CSRC, name)) as f:
            return re.sub(r"//[^\n]*", "", f.read())
    users = [f for f in os.listdir(CSRC) if f.endswith((".cu", ".cuh"))
             and "launch.h" in source(f)]
    assert {"experts.cu", "act_checkpoint.cu", "norm.cu"} <= set(users)
    for name in users + ["rowvec.cuh", "expert_tiles.cuh"]:
        s = source(name)
        assert "__ldg" not in s and "ld.global.nc" not in s, name
        assert not re.search(r"const\s+[\w:]+\s*\*\s*__restrict__", s), name
