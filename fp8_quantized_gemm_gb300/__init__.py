"""Thin Python binding of libfp8gemm.so (the C ABI in include/fp8gemm.h).

Argument marshalling only: each function takes torch CUDA tensors, passes
their device pointers, sizes and the current CUDA stream to the C entry point
of the same name, and raises ``Fp8Error`` on a non-zero status.  Every step of
the computation runs in the library's CUDA kernels; there is no CPU path.

The library must have been built (``python -c "import __graft_entry__ as g;
g.build()"`` or ``python fp8_quantized_gemm_gb300/build.py``); importing this
package without it raises ImportError.
"""
from __future__ import annotations

import ctypes
import os
import struct
import threading

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libfp8gemm.so")

if not os.path.exists(LIB_PATH):
    raise ImportError("libfp8gemm.so is not built (%s); run fp8_quantized_gemm_gb300/build.py" % LIB_PATH)

_lib = ctypes.CDLL(LIB_PATH)

# enums (include/fp8gemm.h)
FP8_OK, FP8_ERR_INVALID_ARG, FP8_ERR_MISALIGNED = 0, -1, -2
FP8_ERR_UNSUPPORTED, FP8_ERR_CUDA, FP8_ERR_TIMEOUT, FP8_ERR_NO_DEVICE = -3, -4, -5, -6
FP8_ERR_SCRATCH_LIMIT = -7
IN_BF16, IN_F32 = 0, 1
E4M3, E5M2 = 0, 1
SCALE_F32, SCALE_UE8M0 = 0, 1
OUT_F32, OUT_BF16 = 0, 1
K_MAJOR, MN_MAJOR = 0, 1
ACT_NONE, ACT_RELU, ACT_RELU2, ACT_SILU, ACT_GELU_TANH, ACT_GELU = 0, 1, 2, 3, 4, 5
NORM_TENSOR, NORM_GROUP, NORM_MX = 0, 1, 2
IDS_I32, IDS_I64 = 0, 1

_vp, _i64, _int, _d = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_double
_SIGS = {
    "fp8_amax": [_vp, _int, _i64, _vp, _vp],
    "fp8_quantize_tensor": [_vp, _int, _i64, _i64, _int, _vp, _vp, _vp, _vp, _vp, _vp, _vp],
    "fp8_quantize_token_group": [_vp, _int, _i64, _i64, _int, _int, _vp, _vp, _vp],
    "fp8_quantize_block": [_vp, _int, _i64, _i64, _int, _int, _vp, _vp, _vp],
    "fp8_quantize_mx": [_vp, _int, _i64, _i64, _int, _vp, _vp, _vp, _vp, _vp],
    "fp8_quantize_mx1": [_vp, _int, _i64, _i64, _int, _vp, _vp, _vp, _vp],
    "fp8_quantize_block32": [_vp, _int, _i64, _i64, _int, _vp, _vp, _vp, _vp],
    "fp8_dequantize_block": [_vp, _int, _vp, _int, _i64, _i64, _vp, _vp],
    "fp8_gemm_tensor": [_vp, _int, _vp, _int, _vp, _vp, _i64, _i64, _i64, _int, _vp, _i64, _int, _vp],
    "fp8_gemm_group": [_vp, _vp, _vp, _vp, _int, _i64, _i64, _i64, _vp, _i64, _vp],
    "fp8_gemm_tensor_grouped": [_vp, _int, _vp],
    "fp8_quantize_tensors": [_vp, _int, _vp, _vp],
    "fp8_gemm_group_experts": [_vp, _vp, _vp, _vp, _int, _vp, _int, _i64, _i64, _i64, _vp, _i64, _vp],
    "fp8_gemm_group_bias": [_vp, _vp, _vp, _vp, _int, _i64, _i64, _i64, _vp, _vp, _i64, _vp],
    "fp8_amax_rows": [_vp, _int, _i64, _i64, _vp, _vp],
    "fp8_quantize_mx_rows": [_vp, _int, _i64, _i64, _int, _vp, _vp, _vp, _vp, _vp],
    "fp8_gemm_mx_rows": [_vp, _vp, _vp, _vp, _vp, _vp, _i64, _i64, _i64, _int, _vp, _i64, _vp],
    "fp8_gemm_mx": [_vp, _vp, _vp, _vp, _vp, _vp, _i64, _i64, _i64, _int, _vp, _i64, _vp],
    "fp8_gemm_group_noalloc": [_vp, _vp, _vp, _vp, _int, _i64, _i64, _i64, _vp, _i64, _vp],
    "fp8_delayed_state_update": [_vp, _vp, _vp, _i64, _int, _vp],
    "fp8_delayed_state_update_multi": [_vp, _int, _vp],
    "fp8_auto_weight_scale": [_vp, _i64, _d, _int, _vp, _vp],
    "fp8_swiglu_forward": [_vp, _vp, _vp, _i64, _vp],
    "fp8_swiglu_backward": [_vp, _vp, _vp, _vp, _vp, _i64, _vp],
    "fp8_adamw_step": [_vp, _vp, _vp, _vp, _vp, _i64, _i64, _d, _d, _d, _d, _d, _vp],
    "fp8_swiglu_forward_quantize": [_vp, _vp, _i64, _int, _vp, _vp, _vp, _vp],
    "fp8_swiglu_backward_quantize": [_vp, _vp, _vp, _i64, _int, _vp, _vp, _vp, _vp, _vp, _vp,
                                     _vp],
    "fp8_adamw_multi": [_vp, _int, _vp, _int, _d, _d, _d, _d, _d, _vp],
    "fp8_quantize_token_group32": [_vp, _int, _i64, _i64, _int, _int, _vp, _vp, _vp],
    "fp8_quantize_block32_f32": [_vp, _int, _i64, _i64, _int, _vp, _vp, _vp],
    "fp8_gemm_group32": [_vp, _vp, _vp, _vp, _i64, _i64, _i64, _vp, _i64, _vp],
    "fp8_rmsnorm_quantize": [_vp, _vp],
    "fp8_rmsnorm_backward": [_vp, _vp],
    "fp8_gemm_tensor_epilogue": [_vp, _vp, _vp],
    "fp8_gemm_tensor_act_backward": [_vp, _vp, _vp],
    "fp8_gemm_group_epilogue": [_vp, _vp, _vp, _vp, _int, _i64, _i64, _i64, _vp, _vp, _vp, _i64,
                                _vp],
    "fp8_experts_sort": [_vp, _int, _i64, _i64, _int, _vp, _vp, _vp, _vp],
    "fp8_experts_gather": [_vp, _vp],
    "fp8_experts_combine": [_vp, _vp],
    "fp8_experts_combine_backward": [_vp, _vp],
    "fp8_act_checkpoint": [_vp, _vp],
    "fp8_act_checkpoint_backward": [_vp, _vp],
    "fp8_get_last_device_error": [ctypes.POINTER(ctypes.c_int), _vp],
    "fp8_set_option": [_int, _int],
}
for _name, _args in _SIGS.items():
    _fn = getattr(_lib, _name)
    _fn.argtypes = _args
    _fn.restype = ctypes.c_int
_lib.fp8_status_string.argtypes = [_int]
_lib.fp8_status_string.restype = ctypes.c_char_p
_lib.fp8_version.argtypes = []
_lib.fp8_version.restype = ctypes.c_char_p

_SIZES = ("fp8_rmsnorm_backward_workspace", "fp8_act_backward_workspace")
for _name in _SIZES:
    _fn = getattr(_lib, _name)
    _fn.argtypes = [_i64, _i64]
    _fn.restype = _i64

EXPORTED = tuple(_SIGS) + _SIZES + ("fp8_status_string", "fp8_version")


class Fp8Error(RuntimeError):
    def __init__(self, name: str, status: int):
        super().__init__("%s failed: %s (%d)" % (name, status_string(status), status))
        self.status = status


def status_string(status: int) -> str:
    return _lib.fp8_status_string(int(status)).decode()


def version() -> str:
    return _lib.fp8_version().decode()


def _p(t):
    """Device pointer of a CUDA tensor (None -> NULL)."""
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("expected a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError("expected a contiguous tensor")
    return t.data_ptr()


def _stream(stream):
    if stream is None:
        return torch.cuda.current_stream().cuda_stream
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _call(name, *args):
    rc = getattr(_lib, name)(*args)
    if rc != FP8_OK:
        raise Fp8Error(name, rc)


def _in_dt(t) -> int:
    if t.dtype == torch.bfloat16:
        return IN_BF16
    if t.dtype == torch.float32:
        return IN_F32
    raise ValueError("input must be bf16 or fp32")


# ----------------------------------------------------------------- calls --

def fp8_amax(x, amax_out, stream=None):
    _call("fp8_amax", _p(x), _in_dt(x), x.numel(), _p(amax_out), _stream(stream))


def fp8_quantize_tensor(x, fmt, q, *, amax_in=None, scale=None, scale_out=None, q_t=None,
                        amax_out=None, stream=None):
    rows, cols = x.shape
    _call("fp8_quantize_tensor", _p(x), _in_dt(x), rows, cols, fmt, _p(amax_in), _p(scale),
          _p(scale_out), _p(q), _p(q_t), _p(amax_out), _stream(stream))


def fp8_quantize_token_group(x, fmt, sfmt, q, scales, stream=None):
    m, k = x.shape
    _call("fp8_quantize_token_group", _p(x), _in_dt(x), m, k, fmt, sfmt, _p(q), _p(scales),
          _stream(stream))


def fp8_quantize_block(w, fmt, sfmt, q, scales, stream=None):
    n, k = w.shape
    _call("fp8_quantize_block", _p(w), _in_dt(w), n, k, fmt, sfmt, _p(q), _p(scales),
          _stream(stream))


def fp8_quantize_mx(x, fmt, amax, global_out, q, local, stream=None):
    r, k = x.shape
    _call("fp8_quantize_mx", _p(x), _in_dt(x), r, k, fmt, _p(amax), _p(global_out), _p(q),
          _p(local), _stream(stream))


def fp8_quantize_mx1(x, fmt, global_out, q, local, stream=None):
    r, k = x.shape
    _call("fp8_quantize_mx1", _p(x), _in_dt(x), r, k, fmt, _p(global_out), _p(q), _p(local),
          _stream(stream))


def fp8_quantize_block32(w, fmt, q, scales, local, stream=None):
    n, k = w.shape
    _call("fp8_quantize_block32", _p(w), _in_dt(w), n, k, fmt, _p(q), _p(scales), _p(local),
          _stream(stream))


def fp8_quantize_token_group32(x, fmt, sfmt, q, scales, stream=None):
    """1x32 token groups; scales group-major [ceil(K/32), M]."""
    m, k = x.shape
    _call("fp8_quantize_token_group32", _p(x), _in_dt(x), m, k, fmt, sfmt, _p(q), _p(scales),
          _stream(stream))


def fp8_quantize_block32_f32(w, fmt, q, scales, stream=None):
    """32x32 weight blocks with fp32 scales [ceil(N/32), K/32]."""
    n, k = w.shape
    _call("fp8_quantize_block32_f32", _p(w), _in_dt(w), n, k, fmt, _p(q), _p(scales),
          _stream(stream))


def fp8_gemm_group32(a, sa, b, sb, out, stream=None):
    """Per-K-group GEMM with fp32 scales of 1x32 groups and 32x32 blocks."""
    m, k = a.shape
    n = b.shape[0]
    _call("fp8_gemm_group32", _p(a), _p(sa), _p(b), _p(sb), m, n, k, _p(out), out.stride(0),
          _stream(stream))


def fp8_dequantize_block(q, fmt, scales, sfmt, out, stream=None):
    n, k = q.shape
    _call("fp8_dequantize_block", _p(q), fmt, _p(scales), sfmt, n, k, _p(out), _stream(stream))


def fp8_gemm_tensor(a, fa, b, fb, sa, sb, out, *, out_dt=None, accumulate=False, stream=None):
    m, k = a.shape
    n = b.shape[0]
    if out_dt is None:
        out_dt = OUT_BF16 if out.dtype == torch.bfloat16 else OUT_F32
    _call("fp8_gemm_tensor", _p(a), fa, _p(b), fb, _p(sa), _p(sb), m, n, k, out_dt, _p(out),
          out.stride(0), int(bool(accumulate)), _stream(stream))


class AdamwEpilogue(ctypes.Structure):
    """fp8_adamw_epilogue_t (include/fp8gemm.h)."""
    _fields_ = [("p", _vp), ("m", _vp), ("v", _vp), ("p_bf16", _vp), ("step", _vp),
                ("lr", _d), ("beta1", _d), ("beta2", _d), ("eps", _d), ("weight_decay", _d)]


class SwigluEpilogue(ctypes.Structure):
    """fp8_swiglu_epilogue_t (include/fp8gemm.h)."""
    _fields_ = [("b_up", _vp), ("sb_up", _vp), ("u", _vp), ("q", _vp), ("fmt", _int),
                ("scale", _vp), ("amax", _vp)]


class GemmProblem(ctypes.Structure):
    """fp8_gemm_problem_t (include/fp8gemm.h)."""
    _fields_ = [("a", _vp), ("b", _vp), ("sa", _vp), ("sb", _vp), ("M", _i64), ("N", _i64),
                ("K", _i64), ("fa", _int), ("fb", _int), ("out_dt", _int), ("accumulate", _int),
                ("c", _vp), ("ldc", _i64), ("a_layout", _int), ("b_layout", _int),
                ("bias", _vp), ("adamw", ctypes.POINTER(AdamwEpilogue)),
                ("swiglu", ctypes.POINTER(SwigluEpilogue))]


def adamw_epilogue(p, m, v, p_bf16, step, lr=1e-4, beta1=0.9, beta2=0.999, eps=1e-8,
                   weight_decay=0.01):
    """AdamW epilogue of a weight-gradient GEMM: the GEMM result (shape of p)
    updates p, m, v and the bf16 copy in place at t = step[0] (device int64,
    read only)."""
    assert step.dtype == torch.int64 and step.numel() == 1
    return AdamwEpilogue(_p(p), _p(m), _p(v), _p(p_bf16), _p(step), lr, beta1, beta2, eps,
                         weight_decay)


def swiglu_epilogue(b_up, sb_up, u, q, fmt, scale, amax):
    """Gated SwiGLU epilogue: the problem's b (W1) and b_up (W3) give h (the
    problem's output) and u; q receives the codes of silu(h) u under `scale`."""
    return SwigluEpilogue(_p(b_up), _p(sb_up), _p(u), _p(q), fmt, _p(scale), _p(amax))


def gemm_problem(a, fa, b, fb, sa, sb, out, *, accumulate=False, a_layout=K_MAJOR,
                 b_layout=K_MAJOR, bias=None, adamw=None, swiglu=None, n=None, ldc=None):
    """Descriptor of one per-tensor GEMM for fp8_gemm_tensor_grouped.  With
    K_MAJOR a is [M, K] and b [N, K]; with MN_MAJOR a is [K, M] and b [K, N];
    bias: optional device fp32 [N] added to every row.  adamw / swiglu:
    epilogue descriptors (adamw_epilogue / swiglu_epilogue); with adamw, `out`
    may be None (the result updates the parameters instead)."""
    m, k = a.shape if a_layout == K_MAJOR else a.shape[::-1]
    if n is None:
        n = b.shape[0] if b_layout == K_MAJOR else b.shape[1]
    if out is None:
        out_dt, c, pitch = OUT_F32, None, ldc if ldc is not None else n
    else:
        out_dt = OUT_BF16 if out.dtype == torch.bfloat16 else OUT_F32
        c, pitch = _p(out), out.stride(0)
    prob = GemmProblem(_p(a), _p(b), _p(sa), _p(sb), m, n, k, fa, fb, out_dt,
                       int(bool(accumulate)), c, pitch, a_layout, b_layout,
                       _p(bias) if bias is not None else None,
                       ctypes.pointer(adamw) if adamw is not None else None,
                       ctypes.pointer(swiglu) if swiglu is not None else None)
    prob._keep = (adamw, swiglu)  # the descriptors live as long as the problem
    return prob


class QuantItem(ctypes.Structure):
    """fp8_quant_item_t (include/fp8gemm.h)."""
    _fields_ = [("x", _vp), ("in_dt", _int), ("n", _i64), ("fmt", _int), ("q", _vp),
                ("amax_out", _vp), ("scale_out", _vp)]


def quant_item(x, fmt, q, scale_out, amax_out=None):
    """Descriptor of one tensor for fp8_quantize_tensors (current scaling)."""
    assert q.numel() == x.numel()
    return QuantItem(_p(x), _in_dt(x), x.numel(), fmt, _p(q),
                     _p(amax_out) if amax_out is not None else None, _p(scale_out))


QUANT_SYNC_WORDS = 8


def fp8_quantize_tensors(items, sync, stream=None):
    """Current scaling of up to four tensors in one launch (pipelined in
    order); `sync` is a device int32 tensor of QUANT_SYNC_WORDS words."""
    assert sync.numel() * sync.element_size() >= 4 * QUANT_SYNC_WORDS
    arr = (QuantItem * len(items))(*items)
    _call("fp8_quantize_tensors", ctypes.cast(arr, _vp), len(items), _p(sync), _stream(stream))


def fp8_gemm_tensor_grouped(problems, stream=None):
    arr = (GemmProblem * len(problems))(*problems)
    _call("fp8_gemm_tensor_grouped", ctypes.cast(arr, _vp), len(problems), _stream(stream))


def fp8_gemm_group(a, sa, b, sb, sfmt, out, stream=None, *, bias=None):
    m, k = a.shape
    n = b.shape[0]
    if bias is not None:
        _call("fp8_gemm_group_bias", _p(a), _p(sa), _p(b), _p(sb), sfmt, m, n, k, _p(bias),
              _p(out), out.stride(0), _stream(stream))
        return
    _call("fp8_gemm_group", _p(a), _p(sa), _p(b), _p(sb), sfmt, m, n, k, _p(out), out.stride(0),
          _stream(stream))


def fp8_gemm_group_experts(a, sa, b, sb, sfmt, offsets, out, stream=None):
    """Per-K-group GEMM of a MoE layer: a [M, K] rows grouped by expert
    (offsets: device int32 [E + 1]), b [E, N, K], sb [E, ceil(N/128), K/128]."""
    m, k = a.shape
    e, n, kb = b.shape
    assert kb == k and offsets.dtype == torch.int32 and offsets.numel() == e + 1
    _call("fp8_gemm_group_experts", _p(a), _p(sa), _p(b), _p(sb), sfmt, _p(offsets), e, m, n, k,
          _p(out), out.stride(0), _stream(stream))


def fp8_gemm_group_noalloc(a, sa, b, sb, sfmt, out, stream=None):
    """fp8_gemm_group without any device allocation (fixed in-library scratch)."""
    m, k = a.shape
    n = b.shape[0]
    _call("fp8_gemm_group_noalloc", _p(a), _p(sa), _p(b), _p(sb), sfmt, m, n, k, _p(out),
          out.stride(0), _stream(stream))


def fp8_gemm_mx(a, la, ga, b, lb, gb, out, *, out_dt=None, stream=None):
    m, k = a.shape
    n = b.shape[0]
    if out_dt is None:
        out_dt = OUT_BF16 if out.dtype == torch.bfloat16 else OUT_F32
    _call("fp8_gemm_mx", _p(a), _p(la), _p(ga), _p(b), _p(lb), _p(gb), m, n, k, out_dt, _p(out),
          out.stride(0), _stream(stream))


def fp8_amax_rows(x, amax_out, stream=None):
    r, k = x.shape
    _call("fp8_amax_rows", _p(x), _in_dt(x), r, k, _p(amax_out), _stream(stream))


def fp8_quantize_mx_rows(x, fmt, amax_rows, global_out, q, local, stream=None):
    r, k = x.shape
    _call("fp8_quantize_mx_rows", _p(x), _in_dt(x), r, k, fmt, _p(amax_rows), _p(global_out),
          _p(q), _p(local), _stream(stream))


def fp8_gemm_mx_rows(a, la, ga, b, lb, gb, out, *, out_dt=None, stream=None):
    m, k = a.shape
    n = b.shape[0]
    if out_dt is None:
        out_dt = OUT_BF16 if out.dtype == torch.bfloat16 else OUT_F32
    _call("fp8_gemm_mx_rows", _p(a), _p(la), _p(ga), _p(b), _p(lb), _p(gb), m, n, k, out_dt,
          _p(out), out.stride(0), _stream(stream))


def fp8_delayed_state_update(hist, scale, amax_cur, fmt, stream=None):
    _call("fp8_delayed_state_update", _p(hist), _p(scale), _p(amax_cur), hist.numel(), fmt,
          _stream(stream))


class DelayedItem(ctypes.Structure):
    """fp8_delayed_item_t (include/fp8gemm.h)."""
    _fields_ = [("hist", _vp), ("scale", _vp), ("amax_cur", _vp), ("L", ctypes.c_int64),
                ("fmt", _int)]


def delayed_item(hist, scale, amax_cur, fmt):
    return DelayedItem(_p(hist), _p(scale), _p(amax_cur), hist.numel(), fmt)


def fp8_delayed_state_update_multi(items, stream=None):
    """Several amax-history steps in one launch (items from delayed_item)."""
    arr = (DelayedItem * len(items))(*items)
    _call("fp8_delayed_state_update_multi", ctypes.cast(arr, ctypes.c_void_p), len(items),
          _stream(stream))


def fp8_auto_weight_scale(amax0, t, lr, fmt, scale_out, stream=None):
    _call("fp8_auto_weight_scale", _p(amax0), int(t), float(lr), fmt, _p(scale_out),
          _stream(stream))


def fp8_swiglu_forward(h, u, a, stream=None):
    _call("fp8_swiglu_forward", _p(h), _p(u), _p(a), h.numel(), _stream(stream))


def fp8_swiglu_backward(da, h, u, dh, du, stream=None):
    _call("fp8_swiglu_backward", _p(da), _p(h), _p(u), _p(dh), _p(du), h.numel(), _stream(stream))


def fp8_adamw_step(p, g, m, v, p_bf16, step, lr=1e-4, beta1=0.9, beta2=0.999, eps=1e-8,
                   weight_decay=0.01, stream=None):
    _call("fp8_adamw_step", _p(p), _p(g), _p(m), _p(v), _p(p_bf16), p.numel(), int(step), lr,
          beta1, beta2, eps, weight_decay, _stream(stream))


def fp8_swiglu_forward_quantize(h, u, fmt, scale, q, amax_out=None, stream=None):
    """a = bf16(silu(h) * u) quantized with the given (delayed) scale into q;
    amax_out receives max |a|.  The bf16 a is not written."""
    assert q.numel() == h.numel() == u.numel()
    _call("fp8_swiglu_forward_quantize", _p(h), _p(u), h.numel(), fmt, _p(scale), _p(q),
          _p(amax_out), _stream(stream))


def fp8_swiglu_backward_quantize(da, h, u, fmt, scale_dh, scale_du, q_dh, q_du, amax_dh=None,
                                 amax_du=None, stream=None):
    """dh, du of a = silu(h) * u, each quantized with its own scale."""
    assert q_dh.numel() == q_du.numel() == h.numel() == u.numel() == da.numel()
    _call("fp8_swiglu_backward_quantize", _p(da), _p(h), _p(u), h.numel(), fmt, _p(scale_dh),
          _p(scale_du), _p(q_dh), _p(q_du), _p(amax_dh), _p(amax_du), _stream(stream))


class AdamwItem(ctypes.Structure):
    """fp8_adamw_item_t (include/fp8gemm.h)."""
    _fields_ = [("p", _vp), ("g", _vp), ("m", _vp), ("v", _vp), ("p_bf16", _vp), ("n", _i64),
                ("q", _vp), ("q_scale", _vp), ("q_amax", _vp), ("q_fmt", _int)]


def adamw_item(p, g, m, v, p_bf16=None, *, q=None, q_scale=None, q_amax=None, q_fmt=E4M3):
    """One tensor of fp8_adamw_multi; with q, also the codes of the updated
    weights (as bf16) under q_scale and their amax (q_amax, nullable)."""
    assert p.numel() == g.numel() == m.numel() == v.numel()
    assert q is None or q.numel() == p.numel()
    return AdamwItem(_p(p), _p(g), _p(m), _p(v), _p(p_bf16), p.numel(), _p(q), _p(q_scale),
                     _p(q_amax), q_fmt)


def fp8_adamw_multi(items, step, lr=1e-4, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.01,
                    stream=None, advance=True):
    """One AdamW step over several tensors; `step` is a device int64 tensor of
    one element, incremented by the call first (the update uses the new
    value) unless advance=False (the update uses it as it stands).  No items:
    only the increment."""
    assert step.dtype == torch.int64 and step.numel() == 1
    arr = (AdamwItem * len(items))(*items) if items else None
    _call("fp8_adamw_multi", ctypes.cast(arr, _vp) if arr is not None else None, len(items),
          _p(step), int(bool(advance)), lr, beta1, beta2, eps, weight_decay, _stream(stream))


# ------------------------------------- RMS norm, linear layer's epilogue --
#
# These calls sit between others on a decoded token's path, where a kernel
# takes a few microseconds: their descriptors are packed with struct (native
# alignment, the C layout) instead of being built field by field, and the
# current stream is read through torch's raw accessor.  ctypes forms of the
# descriptors, for callers that fill them themselves, have the same layout.

class RmsNorm(ctypes.Structure):
    """fp8_rmsnorm_t (include/fp8gemm.h)."""
    _fields_ = [("x", _vp), ("residual", _vp), ("w", _vp), ("dt", _int), ("w_dt", _int),
                ("M", _i64), ("K", _i64), ("ld_x", _i64), ("ld_residual", _i64), ("eps", _d),
                ("mode", _int), ("fmt", _int), ("sfmt", _int), ("scale", _vp), ("q", _vp),
                ("scales", _vp), ("sum_out", _vp), ("ld_sum", _i64), ("y_out", _vp),
                ("ld_y", _i64), ("inv_rms", _vp), ("amax_out", _vp)]


class RmsNormGrad(ctypes.Structure):
    """fp8_rmsnorm_grad_t (include/fp8gemm.h)."""
    _fields_ = [("dy", _vp), ("r", _vp), ("w", _vp), ("d_residual", _vp), ("inv_rms", _vp),
                ("dy_dt", _int), ("dt", _int), ("w_dt", _int), ("M", _i64), ("K", _i64),
                ("ld_dy", _i64), ("ld_r", _i64), ("ld_dres", _i64), ("ld_dx", _i64), ("dx", _vp),
                ("dw", _vp), ("accumulate_dw", _int), ("q", _vp), ("fmt", _int), ("scale", _vp),
                ("amax_out", _vp), ("workspace", _vp), ("workspace_bytes", _i64)]


class LinearEpilogue(ctypes.Structure):
    """fp8_linear_epilogue_t (include/fp8gemm.h)."""
    _fields_ = [("act", _int), ("residual", _vp), ("residual_dt", _int), ("ld_residual", _i64),
                ("pre", _vp), ("ld_pre", _i64), ("q", _vp), ("q_fmt", _int), ("q_scale", _vp),
                ("q_amax", _vp)]


class ActGradEpilogue(ctypes.Structure):
    """fp8_act_grad_epilogue_t (include/fp8gemm.h)."""
    _fields_ = [("act", _int), ("pre", _vp), ("ld_pre", _i64), ("q", _vp), ("q_fmt", _int),
                ("q_scale", _vp), ("q_amax", _vp), ("dbias", _vp), ("accumulate_dbias", _int),
                ("workspace", _vp), ("workspace_bytes", _i64)]


def _packer(cls):
    """struct packer of a descriptor class (checked against its layout)."""
    code = {_vp: "P", _int: "i", _i64: "q", _d: "d"}
    fmt = "@" + "".join(code.get(t, "P") for _, t in cls._fields_) + "0q"
    s = struct.Struct(fmt)
    assert s.size == ctypes.sizeof(cls)
    return s.pack


_pack_norm, _pack_norm_grad = _packer(RmsNorm), _packer(RmsNormGrad)
_pack_epilogue, _pack_act_grad = _packer(LinearEpilogue), _packer(ActGradEpilogue)
_pack_problem = _packer(GemmProblem)
_c_norm, _c_norm_grad = _lib.fp8_rmsnorm_quantize, _lib.fp8_rmsnorm_backward
_c_tensor_epilogue = _lib.fp8_gemm_tensor_epilogue
_c_group_epilogue = _lib.fp8_gemm_group_epilogue
_c_act_backward = _lib.fp8_gemm_tensor_act_backward
_c_norm_grad_ws, _c_act_ws = _lib.fp8_rmsnorm_backward_workspace, _lib.fp8_act_backward_workspace
# (torch's raw accessors where this torch has them: its public functions build
# objects around the same values)
_get_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda dev: torch.cuda.current_stream(dev).cuda_stream)
_stream_of = getattr(torch._C, "_cuda_getCurrentStream", None)
_stream_id = (lambda dev: _stream_of(dev)[0]) if _stream_of else (
    lambda dev: torch.cuda.current_stream(dev).stream_id)
_capturing = getattr(torch._C, "_cuda_isCurrentStreamCapturing", None) or (
    torch.cuda.is_current_stream_capturing)
_BF16, _F32 = torch.bfloat16, torch.float32


def _flat(t):
    """Device pointer of a contiguous CUDA tensor (None -> 0)."""
    if t is None:
        return 0
    if not t.is_cuda or not t.is_contiguous():
        raise ValueError("expected a contiguous CUDA tensor")
    return t.data_ptr()


def _rows(t, shape, dtype, what):
    """(device pointer, row pitch) of a CUDA matrix with contiguous rows, of
    the given shape and type (None -> NULL)."""
    if t is None:
        return 0, 0
    if t.dtype != dtype or t.shape != shape or not t.is_cuda:
        raise ValueError("%s must be a CUDA tensor, %s %s" % (what, dtype, tuple(shape)))
    if t.is_contiguous():
        return t.data_ptr(), shape[1]
    ld, step = t.stride()
    if (step != 1 and shape[1] != 1) or (ld < shape[1] and shape[0] > 1):
        raise ValueError("%s must have contiguous rows" % what)
    return t.data_ptr(), max(ld, shape[1])


def _vector(t, n, what):
    """Device pointer of n contiguous fp32 values (None -> 0)."""
    if t is None:
        return 0
    if t.dtype != _F32 or t.numel() != n or not t.is_cuda or not t.is_contiguous():
        raise ValueError("%s must be contiguous CUDA fp32 [%d]" % (what, n))
    return t.data_ptr()


def _codes(t, n, what):
    if t is None:
        return 0
    if t.element_size() != 1 or t.numel() != n or not t.is_cuda or not t.is_contiguous():
        raise ValueError("%s must hold %d contiguous one-byte CUDA codes" % (what, n))
    return t.data_ptr()


def _scales(t, n, size, what):
    """Device pointer of n scales (or words) of `size` bytes, at least."""
    if t.element_size() != size or t.numel() < n or not t.is_cuda or not t.is_contiguous():
        raise ValueError("%s must hold %d contiguous %d-byte CUDA scales" % (what, n, size))
    return t.data_ptr()


def _gain(w, k):
    """(device pointer, type) of the norm's gains (None: ones)."""
    if w is None:
        return 0, IN_F32
    if w.numel() != k:
        raise ValueError("w must have %d elements" % k)
    return _flat(w), _in_dt(w)


def _on(stream):
    return _raw_stream(_get_device()) if stream is None else _stream(stream)


def _check(name, rc):
    if rc != FP8_OK:
        raise Fp8Error(name, rc)


# Scratch of calls that bring none.  Up to _KEPT bytes come from a buffer kept
# per thread and stream (calls that share it follow one another on that stream;
# allocating it anew costs 3 of a small call's 8 us), as large as the largest of
# these calls needed.  torch's own streams live as long as the process, and their
# ids are odd, or 0 for the default one; any other stream's id is its handle,
# which may be issued again while the work of the stream that had it still runs,
# so its calls keep nothing.  Those, larger ones, and calls recorded into a
# graph, whose memory must live as long as the graph, take theirs from torch's
# allocator in the current stream's order.
_KEPT = 8 << 20
_KEPT_STEP = 64 << 10
_kept = threading.local()


def _scratch(nbytes, workspace, like, stream):
    """(pointer, bytes, owner) of a call's scratch; the owner lives through it.
    like: one of the call's operands, all checked before."""
    if workspace is not None:
        return _flat(workspace), workspace.nbytes, None
    if stream is not None:
        raise ValueError("a call on an explicit stream needs an explicit workspace")
    dev = _get_device()
    if like.device.index != dev:
        raise ValueError("operands must be on the current device")
    if nbytes <= _KEPT and not _capturing():
        sid = _stream_id(dev)
        if sid & 1 or sid == 0:
            try:
                kept = _kept.buffers.get((dev, sid))
            except AttributeError:
                _kept.buffers, kept = {}, None
            if kept is None or kept[1] < nbytes:
                size = max(_KEPT_STEP, 1 << (nbytes - 1).bit_length())
                t = torch.empty(size, dtype=torch.uint8, device=like.device)
                kept = _kept.buffers[dev, sid] = (t.data_ptr(), size, t)
            return kept
    t = torch.empty(nbytes, dtype=torch.uint8, device=like.device)
    return t.data_ptr(), nbytes, t


def fp8_rmsnorm_quantize(x, w, eps, fmt, q, *, residual=None, sum_out=None, scale=None,
                         amax_out=None, scales=None, sfmt=SCALE_F32, local=None, y_out=None,
                         inv_rms=None, stream=None):
    """r = x + residual (-> sum_out), y = r / rms(r) * w (-> y_out, bf16) and
    the codes q of y: per tensor under `scale` (amax_out: max |y|), per 1x128
    group (`scales`, sfmt), or one-level MX (`local` words).  w: [K] gains, or
    None for ones; inv_rms: fp32 [M], kept for fp8_rmsnorm_backward."""
    shape, t = x.shape, x.dtype
    m, k = shape
    if (scale is not None) + (scales is not None) + (local is not None) != 1:
        raise ValueError("one of scale, scales and local selects the quantization")
    px, ldx = _rows(x, shape, t, "x")
    pr, ldr = _rows(residual, shape, t, "residual")
    ps, lds = _rows(sum_out, shape, t, "sum_out")
    py, ldy = _rows(y_out, shape, _BF16, "y_out")
    pw, wdt = _gain(w, k)
    if scale is not None:
        mode, psc = NORM_TENSOR, 0
    elif scales is not None:
        mode = NORM_GROUP
        psc = _scales(scales, (k + 127) // 128 * m, 4 if sfmt == SCALE_F32 else 1, "scales")
    else:
        mode, psc = NORM_MX, _scales(local, k // 128 * ((m + 127) // 128 * 128), 4, "local")
    d = _pack_norm(px, pr, pw, _in_dt(x), wdt, m, k, ldx, ldr, eps, mode, fmt, sfmt,
                   _vector(scale, 1, "scale"), _codes(q, m * k, "q"), psc, ps, lds, py, ldy,
                   _vector(inv_rms, m, "inv_rms"), _vector(amax_out, 1, "amax_out"))
    _check("fp8_rmsnorm_quantize", _c_norm(d, _on(stream)))


def fp8_rmsnorm_backward_workspace(m, k):
    """Bytes of scratch that fp8_rmsnorm_backward needs for dw."""
    return _lib.fp8_rmsnorm_backward_workspace(m, k)


def fp8_rmsnorm_backward(dy, r, inv_rms, w, dx, *, d_residual=None, dw=None, accumulate_dw=False,
                         q=None, fmt=E5M2, scale=None, amax_out=None, workspace=None, stream=None):
    """dx = gradient of x and of residual, through the norm and (d_residual)
    past it; dw: fp32 [K]; q: the codes of dx under `scale`, amax_out its
    max |dx|.  r, inv_rms: as fp8_rmsnorm_quantize wrote them.  workspace
    (with dw): device scratch; None: the binding's own."""
    shape, t = r.shape, r.dtype
    m, k = shape
    py, ldy = _rows(dy, shape, dy.dtype, "dy")
    pr, ldr = _rows(r, shape, t, "r")
    pe, lde = _rows(d_residual, shape, t, "d_residual")
    px, ldx = _rows(dx, shape, t, "dx")
    pw, wdt = _gain(w, k)
    pi, pdw, pq = _vector(inv_rms, m, "inv_rms"), _vector(dw, k, "dw"), _codes(q, m * k, "q")
    ps, pa = _vector(scale, 1, "scale"), _vector(amax_out, 1, "amax_out")
    pws, ws_bytes, keep = (0, 0, None) if dw is None else _scratch(
        _c_norm_grad_ws(m, k), workspace, r, stream)
    d = _pack_norm_grad(py, pr, pw, pe, pi, _in_dt(dy), _in_dt(r), wdt, m, k, ldy, ldr, lde, ldx,
                        px, pdw, int(bool(accumulate_dw)), pq, fmt, ps, pa, pws, ws_bytes)
    _check("fp8_rmsnorm_backward", _c_norm_grad(d, _on(stream)))


def _epilogue_problem(a, fa, b, fb, sa, sb, out, a_layout, b_layout, bias):
    """(M, N) shape and packed fp8_gemm_problem_t of an epilogue call."""
    m, k = a.shape
    n, kb = b.shape
    if a_layout != K_MAJOR:
        m, k = k, m
    if b_layout != K_MAJOR:
        n, kb = kb, n
    if kb != k:
        raise ValueError("operands of different K")
    shape = (m, n)
    dt = OUT_BF16 if out is None or out.dtype == _BF16 else OUT_F32
    c, ldc = _rows(out, shape, _BF16 if dt == OUT_BF16 else _F32, "out")
    return shape, _pack_problem(
        _codes(a, m * k, "a"), _codes(b, n * k, "b"), _vector(sa, 1, "sa"), _vector(sb, 1, "sb"),
        m, n, k, fa, fb, dt, 0, c, ldc, a_layout, b_layout, _vector(bias, n, "bias"), 0, 0)


def _linear_epilogue(shape, act, residual, pre_out, q=None, q_fmt=E4M3, q_scale=None, q_amax=None):
    f32 = residual is not None and residual.dtype == _F32
    pr, ldr = _rows(residual, shape, _F32 if f32 else _BF16, "residual")
    pp, ldp = _rows(pre_out, shape, _BF16, "pre_out")
    return _pack_epilogue(act, pr, OUT_F32 if f32 else OUT_BF16, ldr, pp, ldp,
                          _codes(q, shape[0] * shape[1], "q"), q_fmt,
                          _vector(q_scale, 1, "q_scale"), _vector(q_amax, 1, "q_amax"))


def fp8_gemm_tensor_epilogue(a, fa, b, fb, sa, sb, out, *, bias=None, act=ACT_NONE, residual=None,
                             pre_out=None, q=None, q_fmt=E4M3, q_scale=None, q_amax=None,
                             a_layout=K_MAJOR, b_layout=K_MAJOR, stream=None):
    """Per-tensor GEMM with y = act(z) + residual, z = sa sb A B^T + bias, in
    its epilogue: out (bf16, fp32, or None with q) <- y, pre_out <- bf16(z),
    q <- codes of y under q_scale, q_amax <- max |y|."""
    shape, p = _epilogue_problem(a, fa, b, fb, sa, sb, out, a_layout, b_layout, bias)
    e = _linear_epilogue(shape, act, residual, pre_out, q, q_fmt, q_scale, q_amax)
    _check("fp8_gemm_tensor_epilogue", _c_tensor_epilogue(p, e, _on(stream)))


def fp8_gemm_group_epilogue(a, sa, b, sb, sfmt, out, *, bias=None, act=ACT_NONE, residual=None,
                            pre_out=None, stream=None):
    """Per-K-group GEMM with the same epilogue; out bf16."""
    m, k = a.shape
    n = b.shape[0]
    shape = (m, n)
    e = _linear_epilogue(shape, act, residual, pre_out)
    c, ldc = _rows(out, shape, _BF16, "out")
    g, size = k // 128, 4 if sfmt == SCALE_F32 else 1
    _check("fp8_gemm_group_epilogue",
           _c_group_epilogue(_codes(a, m * k, "a"), _scales(sa, g * m, size, "sa"),
                             _codes(b, n * k, "b"), _scales(sb, (n + 127) // 128 * g, size, "sb"),
                             sfmt, m, n, k, _vector(bias, n, "bias"), e, c, ldc, _on(stream)))


def fp8_act_backward_workspace(m, n):
    """Bytes of scratch that fp8_gemm_tensor_act_backward needs for dbias."""
    return _lib.fp8_act_backward_workspace(m, n)


def fp8_gemm_tensor_act_backward(a, fa, b, fb, sa, sb, pre, act, *, out=None, q=None, q_fmt=E5M2,
                                 q_scale=None, q_amax=None, dbias=None, accumulate_dbias=False,
                                 workspace=None, a_layout=K_MAJOR, b_layout=K_MAJOR, stream=None):
    """dz = (sa sb A B^T) * act'(pre) in the GEMM's epilogue: out (bf16 or
    fp32) and/or q <- codes of dz under q_scale (q_amax: max |dz|); dbias:
    fp32 [N] column sums.  workspace (with dbias): device scratch; None: the
    binding's own."""
    shape, p = _epilogue_problem(a, fa, b, fb, sa, sb, out, a_layout, b_layout, None)
    m, n = shape
    pp, ldp = _rows(pre, shape, _BF16, "pre")
    pq, ps = _codes(q, m * n, "q"), _vector(q_scale, 1, "q_scale")
    pa, pdb = _vector(q_amax, 1, "q_amax"), _vector(dbias, n, "dbias")
    pws, ws_bytes, keep = (0, 0, None) if dbias is None else _scratch(
        _c_act_ws(m, n), workspace, pre, stream)
    e = _pack_act_grad(act, pp, ldp, pq, q_fmt, ps, pa, pdb, int(bool(accumulate_dbias)), pws,
                       ws_bytes)
    _check("fp8_gemm_tensor_act_backward", _c_act_backward(p, e, _on(stream)))


# ------------------- tokens to their experts and back, 8-bit checkpoints --

class ExpertsGather(ctypes.Structure):
    """fp8_experts_gather_t (include/fp8gemm.h)."""
    _fields_ = [("x", _vp), ("dt", _int), ("ld_x", _i64), ("xq", _vp), ("x_scales", _vp),
                ("rows", _vp), ("T", _i64), ("S", _i64), ("K", _i64), ("M", _i64), ("fmt", _int),
                ("sfmt", _int), ("q", _vp), ("scales", _vp), ("out", _vp), ("ld_out", _i64)]


class ExpertsCombine(ctypes.Structure):
    """fp8_experts_combine_t (include/fp8gemm.h)."""
    _fields_ = [("x", _vp), ("x_dt", _int), ("ld_x", _i64), ("rows", _vp), ("weights", _vp),
                ("T", _i64), ("S", _i64), ("K", _i64), ("M", _i64), ("residual", _vp),
                ("ld_residual", _i64), ("out", _vp), ("out_dt", _int), ("ld_out", _i64)]


class ExpertsCombineGrad(ctypes.Structure):
    """fp8_experts_combine_grad_t (include/fp8gemm.h)."""
    _fields_ = [("dy", _vp), ("dy_dt", _int), ("ld_dy", _i64), ("x", _vp), ("x_dt", _int),
                ("ld_x", _i64), ("rows", _vp), ("weights", _vp), ("T", _i64), ("S", _i64),
                ("K", _i64), ("M", _i64), ("d_weights", _vp), ("q", _vp), ("scales", _vp),
                ("fmt", _int), ("sfmt", _int), ("dx", _vp), ("dx_dt", _int), ("ld_dx", _i64)]


class ActCheckpoint(ctypes.Structure):
    """fp8_act_checkpoint_t (include/fp8gemm.h)."""
    _fields_ = [("act", _int), ("h", _vp), ("ld_h", _i64), ("u", _vp), ("ld_u", _i64),
                ("M", _i64), ("N", _i64), ("valid_rows", _vp), ("mode", _int), ("fmt", _int),
                ("sfmt", _int), ("q", _vp), ("scale", _vp), ("scales", _vp), ("amax_out", _vp),
                ("keep_sfmt", _int), ("h_q", _vp), ("h_scales", _vp), ("u_q", _vp),
                ("u_scales", _vp), ("out", _vp), ("ld_out", _i64)]


class ActCheckpointGrad(ctypes.Structure):
    """fp8_act_checkpoint_grad_t (include/fp8gemm.h)."""
    _fields_ = [("act", _int), ("da", _vp), ("ld_da", _i64), ("h_q", _vp), ("h_scales", _vp),
                ("u_q", _vp), ("u_scales", _vp), ("keep_sfmt", _int), ("M", _i64), ("N", _i64),
                ("valid_rows", _vp), ("mode", _int), ("fmt", _int), ("sfmt", _int), ("dh_q", _vp),
                ("du_q", _vp), ("ld_q", _i64), ("scale_dh", _vp), ("scale_du", _vp),
                ("dh_scales", _vp), ("du_scales", _vp), ("amax_dh", _vp), ("amax_du", _vp),
                ("dh", _vp), ("du", _vp), ("ld_d", _i64)]


_pack_gather, _pack_combine = _packer(ExpertsGather), _packer(ExpertsCombine)
_pack_combine_grad = _packer(ExpertsCombineGrad)
_pack_act, _pack_act_ckpt_grad = _packer(ActCheckpoint), _packer(ActCheckpointGrad)
_c_sort, _c_gather = _lib.fp8_experts_sort, _lib.fp8_experts_gather
_c_combine, _c_combine_grad = _lib.fp8_experts_combine, _lib.fp8_experts_combine_backward
_c_act, _c_act_grad = _lib.fp8_act_checkpoint, _lib.fp8_act_checkpoint_backward
_I32, _I64, _U8 = torch.int32, torch.int64, torch.uint8


# Checks of one operand each, for calls that sit between decoded tokens' kernels:
# an attribute of a tensor costs 0.06 to 0.12 us here, a kernel two to three, so
# each is read once (get_device() is -1 off the GPU and so covers is_cuda).

def _matrix(t, m, n, dtype, dev, what):
    """(device pointer, row pitch) of a matrix [m, n] with contiguous rows."""
    if t.dtype is dtype and t.get_device() == dev and t.shape == (m, n):
        ld, one = t.stride()
        if m == 1 and one == 1:
            return t.data_ptr(), n
        if one == 1 and ld >= n:
            return t.data_ptr(), ld
        if m == 0:
            return 0, n
    raise ValueError("%s must be a matrix of %s [%d, %d] with contiguous rows on the current device"
                     % (what, dtype, m, n))


def _list(t, dtype, n, dev, what):
    """Device pointer of n contiguous values."""
    if t.dtype is dtype and t.numel() == n and t.get_device() == dev and t.is_contiguous():
        return t.data_ptr()
    raise ValueError("%s must be contiguous %s [%d] on the current device" % (what, dtype, n))


def _group_codes(q, scales, m, k, sfmt, dev, what):
    """Device pointers of codes [m, k] and their 1x128-group scales."""
    if q is None or scales is None:
        raise ValueError("%s needs its scales, and they it" % what)
    if (q.element_size() != 1 or q.numel() != m * k or q.get_device() != dev
            or not q.is_contiguous()):
        raise ValueError("%s must hold %d contiguous one-byte codes on the current device"
                         % (what, m * k))
    return q.data_ptr(), _group_scales(scales, m, k, sfmt, dev, what)


def _group_scales(scales, m, k, sfmt, dev, what):
    """Device pointer of the scales of [m, k] in 1x128 groups, at least."""
    size = 4 if sfmt == SCALE_F32 else 1
    if (scales.element_size() != size or scales.numel() < (k + 127) // 128 * m
            or scales.get_device() != dev or not scales.is_contiguous()):
        raise ValueError("%s's scales must be %d contiguous %d-byte values on the current device"
                         % (what, (k + 127) // 128 * m, size))
    return scales.data_ptr()


def _float_type(t, what):
    if t.dtype is _BF16:
        return IN_BF16
    if t.dtype is _F32:
        return IN_F32
    raise ValueError("%s must be bf16 or fp32" % what)


def fp8_experts_sort(ids, experts, offsets, rows, pairs=None, stream=None):
    """Rows in expert order of the choices ids [T, S] (int32 or int64): offsets
    int32 [experts + 1], rows int32 [T, S] (-1: dropped, an id outside
    [0, experts)), pairs (optional) int32 [T * S], -1 behind the last row."""
    dev = _get_device()
    t, s = ids.shape
    n = t * s
    if ids.dtype is _I64:
        dt = IDS_I64
    elif ids.dtype is _I32:
        dt = IDS_I32
    else:
        raise ValueError("ids must be int32 or int64")
    rc = _c_sort(_list(ids, ids.dtype, n, dev, "ids"), dt, t, s, experts,
                 _list(offsets, _I32, experts + 1, dev, "offsets"),
                 _list(rows, _I32, n, dev, "rows"),
                 0 if pairs is None else _list(pairs, _I32, n, dev, "pairs"),
                 _raw_stream(dev) if stream is None else _stream(stream))
    if rc:
        raise Fp8Error("fp8_experts_sort", rc)


def fp8_experts_gather(x, rows, *, q=None, scales=None, fmt=E4M3, sfmt=SCALE_F32, x_scales=None,
                       out=None, stream=None):
    """Row rows[t, s] <- x[t]: as 1x128-group codes (q [M, K] with scales
    [ceil(K/128), M]) and / or as it is (out [M, K] of x's type).  x bf16 or
    fp32, or codes with x_scales [ceil(K/128), T], which are moved."""
    dev = _get_device()
    t, k = x.shape
    if rows.dim() != 2 or rows.shape[0] != t:
        raise ValueError("rows must be [T, S]")
    n = rows.numel()
    m = _grouped_rows(out if q is None else q, k, "q or out")
    pq = ps = po = ldo = px = ldx = dt = pc = pcs = 0
    if q is not None or scales is not None:
        pq, ps = _group_codes(q, scales, m, k, sfmt, dev, "q")
    if x_scales is not None:
        if out is not None:
            raise ValueError("codes are moved into q")
        pc, pcs = _group_codes(x, x_scales, t, k, sfmt, dev, "x")
    else:
        dt = _float_type(x, "x")
        px, ldx = _matrix(x, t, k, x.dtype, dev, "x")
        if out is not None:
            po, ldo = _matrix(out, m, k, x.dtype, dev, "out")
    rc = _c_gather(_pack_gather(px, dt, ldx, pc, pcs, _list(rows, _I32, n, dev, "rows"), t,
                                rows.shape[1], k, m, fmt, sfmt, pq, ps, po, ldo),
                   _raw_stream(dev) if stream is None else _stream(stream))
    if rc:
        raise Fp8Error("fp8_experts_gather", rc)


def _grouped_rows(t, k, what):
    """Rows of the grouped side: M of a matrix [M, k]."""
    if t is None:
        raise ValueError("%s takes the rows" % what)
    m, kt = t.shape
    if kt != k:
        raise ValueError("%s must be [M, %d]" % (what, k))
    return m


def _weights(weights, rows, n, dev):
    if weights is None:
        return 0
    if weights.shape != rows.shape:
        raise ValueError("weights must have the shape of rows")
    return _list(weights, _F32, n, dev, "weights")


def fp8_experts_combine(x, rows, weights, out, *, residual=None, stream=None):
    """out[t] = residual[t] + sum_s weights[t, s] x[rows[t, s]] (weights None:
    ones, the gradient of fp8_experts_gather).  x [M, K], out and residual
    [T, K]: bf16 or fp32."""
    dev = _get_device()
    t, s = rows.shape
    m, k = x.shape
    n = t * s
    xdt, odt = _float_type(x, "x"), _float_type(out, "out")
    px, ldx = _matrix(x, m, k, x.dtype, dev, "x")
    po, ldo = _matrix(out, t, k, out.dtype, dev, "out")
    pr = ldr = 0
    if residual is not None:
        pr, ldr = _matrix(residual, t, k, out.dtype, dev, "residual")
    rc = _c_combine(_pack_combine(px, xdt, ldx, _list(rows, _I32, n, dev, "rows"),
                                  _weights(weights, rows, n, dev), t, s, k, m, pr, ldr, po, odt,
                                  ldo),
                    _raw_stream(dev) if stream is None else _stream(stream))
    if rc:
        raise Fp8Error("fp8_experts_combine", rc)


def fp8_experts_combine_backward(dy, rows, weights, *, x=None, d_weights=None, q=None, scales=None,
                                 fmt=E4M3, sfmt=SCALE_F32, dx=None, stream=None):
    """The gradient of fp8_experts_combine: row rows[t, s] of q (1x128-group
    codes with scales) and / or dx (bf16 or fp32) <- weights[t, s] dy[t];
    d_weights fp32 [T, S] <- <dy[t], x[rows[t, s]]> (x: what combine read)."""
    dev = _get_device()
    t, s = rows.shape
    n, k = t * s, dy.shape[1]
    m = _grouped_rows(q if q is not None else dx if dx is not None else x, k, "q, dx or x")
    ddt = _float_type(dy, "dy")
    pdy, ldy = _matrix(dy, t, k, dy.dtype, dev, "dy")
    px = ldx = pdx = lddx = pq = ps = pdw = 0
    xdt = dxdt = IN_BF16
    if x is not None:
        xdt = _float_type(x, "x")
        px, ldx = _matrix(x, m, k, x.dtype, dev, "x")
    if d_weights is not None:
        if x is None:
            raise ValueError("d_weights needs x")
        pdw = _list(d_weights, _F32, n, dev, "d_weights")
    if dx is not None:
        dxdt = _float_type(dx, "dx")
        pdx, lddx = _matrix(dx, m, k, dx.dtype, dev, "dx")
    if q is not None or scales is not None:
        pq, ps = _group_codes(q, scales, m, k, sfmt, dev, "q")
    rc = _c_combine_grad(
        _pack_combine_grad(pdy, ddt, ldy, px, xdt, ldx, _list(rows, _I32, n, dev, "rows"),
                           _weights(weights, rows, n, dev), t, s, k, m, pdw, pq, ps, fmt, sfmt,
                           pdx, dxdt, lddx),
        _raw_stream(dev) if stream is None else _stream(stream))
    if rc:
        raise Fp8Error("fp8_experts_combine_backward", rc)


def fp8_act_checkpoint(h, u, act, q, *, fmt=E4M3, scale=None, amax_out=None, scales=None,
                       sfmt=SCALE_F32, h_q=None, h_scales=None, u_q=None, u_scales=None,
                       keep_sfmt=SCALE_F32, out=None, valid_rows=None, stream=None):
    """q <- codes of a = act(h) u (u None: act(h)), per tensor under `scale`
    (amax_out: max |a|) or per 1x128 group (scales, sfmt); h_q, u_q (both or
    neither) <- the checkpoints of h and u: E4M3 codes with 1x128-group scales
    of keep_sfmt; out: a in bf16.  valid_rows: device int32, rows from it on
    are left alone."""
    dev = _get_device()
    m, n = h.shape
    ph, ldh = _matrix(h, m, n, _BF16, dev, "h")
    pu = ldu = po = ldo = ps = psc = pa = phq = phs = puq = pus = pv = 0
    if u is not None:
        pu, ldu = _matrix(u, m, n, _BF16, dev, "u")
    if scale is not None:
        if scales is not None:
            raise ValueError("one of scale and scales selects the quantization")
        mode, psc = NORM_TENSOR, _list(scale, _F32, 1, dev, "scale")
        if (q.element_size() != 1 or q.numel() != m * n or q.get_device() != dev
                or not q.is_contiguous()):
            raise ValueError("q must hold %d contiguous one-byte codes on the current device"
                             % (m * n))
        pq = q.data_ptr()
        if amax_out is not None:
            pa = _list(amax_out, _F32, 1, dev, "amax_out")
    elif scales is not None:
        mode = NORM_GROUP
        pq, ps = _group_codes(q, scales, m, n, sfmt, dev, "q")
        if amax_out is not None:
            raise ValueError("amax_out goes with scale")
    else:
        raise ValueError("one of scale and scales selects the quantization")
    if h_q is not None or h_scales is not None:
        phq, phs = _group_codes(h_q, h_scales, m, n, keep_sfmt, dev, "h_q")
    if u_q is not None or u_scales is not None:
        puq, pus = _group_codes(u_q, u_scales, m, n, keep_sfmt, dev, "u_q")
    if out is not None:
        po, ldo = _matrix(out, m, n, _BF16, dev, "out")
    if valid_rows is not None:
        pv = _list(valid_rows, _I32, 1, dev, "valid_rows")
    rc = _c_act(_pack_act(act, ph, ldh, pu, ldu, m, n, pv, mode, fmt, sfmt, pq, psc, ps, pa,
                          keep_sfmt, phq, phs, puq, pus, po, ldo),
                _raw_stream(dev) if stream is None else _stream(stream))
    if rc:
        raise Fp8Error("fp8_act_checkpoint", rc)


def _code_rows(t, m, n, dev, what):
    """(device pointer, row pitch in bytes) of codes with contiguous rows."""
    if t.element_size() != 1:
        raise ValueError("%s must hold one-byte codes" % what)
    return _matrix(t, m, n, t.dtype, dev, what)


def fp8_act_checkpoint_backward(da, act, h_q, h_scales, u_q=None, u_scales=None, *,
                                keep_sfmt=SCALE_F32, dh_q=None, du_q=None, fmt=E5M2,
                                scale_dh=None, scale_du=None, amax_dh=None, amax_du=None,
                                dh_scales=None, du_scales=None, sfmt=SCALE_F32, dh=None, du=None,
                                valid_rows=None, stream=None):
    """dh = da u act'(h), du = da act(h) at the values of fp8_act_checkpoint's
    checkpoints (u_q None: no gate): codes dh_q, du_q of one row pitch, per
    tensor (scale_dh, scale_du, amaxes) or per 1x128 group (dh_scales,
    du_scales, sfmt), and / or dh, du in bf16 (of one row pitch)."""
    dev = _get_device()
    m, n = da.shape
    pda, ldda = _matrix(da, m, n, _BF16, dev, "da")
    phq, phs = _group_codes(h_q, h_scales, m, n, keep_sfmt, dev, "h_q")
    puq = pus = pqh = pqu = ldq = psh = psu = psch = pscu = pah = pau = pdh = pdu = ldd = pv = 0
    if u_q is not None or u_scales is not None:
        puq, pus = _group_codes(u_q, u_scales, m, n, keep_sfmt, dev, "u_q")
    if dh_q is not None:
        pqh, ldq = _code_rows(dh_q, m, n, dev, "dh_q")
    if du_q is not None:
        pqu, ld = _code_rows(du_q, m, n, dev, "du_q")
        if dh_q is not None and ld != ldq:
            raise ValueError("dh_q and du_q must have one row pitch")
        ldq = ld
    if dh_scales is not None or du_scales is not None:
        mode = NORM_GROUP
        if (scale_dh is not None or scale_du is not None or amax_dh is not None
                or amax_du is not None):
            raise ValueError("scales per tensor or per group, not both")
        if (dh_q is None) != (dh_scales is None) or (du_q is None) != (du_scales is None):
            raise ValueError("codes need their scales, and they them")
        if dh_q is not None:
            psh = _group_scales(dh_scales, m, n, sfmt, dev, "dh_q")
        if du_q is not None:
            psu = _group_scales(du_scales, m, n, sfmt, dev, "du_q")
    else:
        mode = NORM_TENSOR
        if scale_dh is not None:
            psch = _list(scale_dh, _F32, 1, dev, "scale_dh")
        if scale_du is not None:
            pscu = _list(scale_du, _F32, 1, dev, "scale_du")
        if amax_dh is not None:
            pah = _list(amax_dh, _F32, 1, dev, "amax_dh")
        if amax_du is not None:
            pau = _list(amax_du, _F32, 1, dev, "amax_du")
    if dh is not None:
        pdh, ldd = _matrix(dh, m, n, _BF16, dev, "dh")
    if du is not None:
        pdu, ld = _matrix(du, m, n, _BF16, dev, "du")
        if dh is not None and ld != ldd:
            raise ValueError("dh and du must have one row pitch")
        ldd = ld
    if valid_rows is not None:
        pv = _list(valid_rows, _I32, 1, dev, "valid_rows")
    rc = _c_act_grad(
        _pack_act_ckpt_grad(act, pda, ldda, phq, phs, puq, pus, keep_sfmt, m, n, pv, mode, fmt,
                            sfmt, pqh, pqu, ldq, psch, pscu, psh, psu, pah, pau, pdh, pdu, ldd),
        _raw_stream(dev) if stream is None else _stream(stream))
    if rc:
        raise Fp8Error("fp8_act_checkpoint_backward", rc)


def fp8_get_last_device_error(stream=None):
    """(status, where): status 0 or FP8_ERR_TIMEOUT; clears the word."""
    where = ctypes.c_int(0)
    rc = _lib.fp8_get_last_device_error(ctypes.byref(where), _stream(stream))
    return rc, where.value


(OPT_GEMM_CTA_PAIRS, OPT_WAIT_LIMIT_US, OPT_GEMM_MULTICAST, OPT_GEMM_TMA_STORE,
 OPT_GEMM_FEW_ROWS, OPT_GEMM_BAND_ROWS, OPT_GEMM_SKINNY) = 1, 2, 3, 4, 5, 6, 7


def fp8_set_option(option, value):
    _call("fp8_set_option", int(option), int(value))


# ------------------------------------------------------------ allocation --

def mx_local_words(rows: int, k: int, device="cuda"):
    """Buffer for fp8_quantize_mx's packed local factors: uint32 [K/128, R_pad]."""
    rpad = (rows + 127) // 128 * 128
    return torch.empty((k // 128, rpad), dtype=torch.int32, device=device)
