// C entry points of the operators around the experts' products: tokens to
// their experts' rows and back, and the activation checkpointed in 8 bits.
// Argument checks and launches.
#include <nvtx3/nvToolsExt.h>

#include "act_checkpoint.h"
#include "experts.h"
#include "fp8gemm.h"
#include "kernels.h"

namespace fp8k {
int api_device(int *sms, uint32_t **err);
}  // namespace fp8k

namespace {

constexpr int64_t kMaxDim = (int64_t)1 << 31;

struct NvtxRange {
  explicit NvtxRange(const char *name) { nvtxRangePushA(name); }
  ~NvtxRange() { nvtxRangePop(); }
  NvtxRange(const NvtxRange &) = delete;
  NvtxRange &operator=(const NvtxRange &) = delete;
};

int to_status(cudaError_t e) { return e == cudaSuccess ? FP8_OK : FP8_ERR_CUDA; }
bool aligned_to(const void *p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
bool valid_in(int d) { return d == FP8_IN_BF16 || d == FP8_IN_F32; }
bool valid_fmt(int f) { return f == FP8_E4M3 || f == FP8_E5M2; }
bool valid_sfmt(int f) { return f == FP8_SCALE_F32 || f == FP8_SCALE_UE8M0; }
bool scales_aligned(const void *p, int sfmt) { return aligned_to(p, sfmt == FP8_SCALE_F32 ? 4 : 1); }

int sm_count(int *sms) {
  uint32_t *err = nullptr;
  return fp8k::api_device(sms, &err);
}

// A nullable matrix read and written in 16-byte vectors of eight elements.
int check_rows(const void *p, int64_t ld, int64_t cols) {
  if (p == nullptr) return FP8_OK;
  if (ld < cols || ld >= kMaxDim) return FP8_ERR_INVALID_ARG;
  return aligned_to(p, 16) && ld % 8 == 0 ? FP8_OK : FP8_ERR_MISALIGNED;
}

// The same for the expert-row calls, whose kernels keep a row's bytes in 32 bits.
int check_expert_rows(const void *p, int64_t ld, int64_t cols) {
  const int rc = check_rows(p, ld, cols);
  return rc == FP8_OK && p != nullptr && ld >= kMaxDim / 2 ? FP8_ERR_UNSUPPORTED : rc;
}

// The sizes of the expert-row calls.
int check_tokens(int64_t T, int64_t S, int64_t K, int64_t M, const int32_t *rows) {
  if (T < 0 || S < 1 || K < 1 || M < 0) return FP8_ERR_INVALID_ARG;
  if (T >= kMaxDim || S >= kMaxDim || K >= kMaxDim || M >= kMaxDim || T * S >= kMaxDim)
    return FP8_ERR_INVALID_ARG;
  if (T > 0 && rows == nullptr) return FP8_ERR_INVALID_ARG;
  if (K % 16 != 0 || !aligned_to(rows, 4)) return FP8_ERR_MISALIGNED;
  return FP8_OK;
}

// combine and its gradient step through a token's choices in 32 signed bits, up to
// eight behind the last one.
int check_choices(int64_t S) { return S > kMaxDim / 2 ? FP8_ERR_UNSUPPORTED : FP8_OK; }

}  // namespace

extern "C" {

int fp8_experts_sort(const void *ids, int id_dt, int64_t T, int64_t S, int experts,
                     int32_t *offsets, int32_t *rows, int32_t *pairs, fp8_stream_t stream) {
  const NvtxRange nvtx_range(__func__);
  if (id_dt != FP8_IDS_I32 && id_dt != FP8_IDS_I64) return FP8_ERR_INVALID_ARG;
  if (T < 0 || S < 1 || T >= kMaxDim || S >= kMaxDim || T * S >= kMaxDim) return FP8_ERR_INVALID_ARG;
  if (experts < 1 || experts > fp8k::kMaxExperts) return FP8_ERR_INVALID_ARG;
  if (offsets == nullptr || (T > 0 && (ids == nullptr || rows == nullptr))) return FP8_ERR_INVALID_ARG;
  // the ranks wait in rows while ids are read again
  if (rows != nullptr && (rows == ids || rows == pairs || rows == offsets)) return FP8_ERR_INVALID_ARG;
  if (!aligned_to(ids, id_dt == FP8_IDS_I64 ? 8 : 4) || !aligned_to(offsets, 4) ||
      !aligned_to(rows, 4) || !aligned_to(pairs, 4))
    return FP8_ERR_MISALIGNED;
  int sms = 0;
  const int rc = sm_count(&sms);
  if (rc != FP8_OK) return rc;
  return to_status(fp8k::launch_experts_sort(ids, id_dt == FP8_IDS_I64, T * S, experts, offsets,
                                             rows, pairs, (cudaStream_t)stream));
}

int fp8_experts_gather(const fp8_experts_gather_t *gather, fp8_stream_t stream) {
  const NvtxRange nvtx_range(__func__);
  if (gather == nullptr) return FP8_ERR_INVALID_ARG;
  const fp8_experts_gather_t &n = *gather;
  int rc = check_tokens(n.T, n.S, n.K, n.M, n.rows);
  if (rc != FP8_OK) return rc;
  const bool codes = n.xq != nullptr;
  if (codes && (n.x != nullptr || n.out != nullptr)) return FP8_ERR_UNSUPPORTED;
  if (!valid_fmt(n.fmt) || !valid_sfmt(n.sfmt) || (!codes && !valid_in(n.dt)))
    return FP8_ERR_INVALID_ARG;
  if ((n.q == nullptr) != (n.scales == nullptr)) return FP8_ERR_INVALID_ARG;
  if (n.T > 0 && n.M > 0) {
    if (!codes && n.x == nullptr) return FP8_ERR_INVALID_ARG;
    if (codes && (n.x_scales == nullptr || n.q == nullptr)) return FP8_ERR_INVALID_ARG;
    if (n.q == nullptr && n.out == nullptr) return FP8_ERR_INVALID_ARG;
  }
  if (!codes && (rc = check_expert_rows(n.x, n.ld_x, n.K)) != FP8_OK) return rc;
  if ((rc = check_expert_rows(n.out, n.ld_out, n.K)) != FP8_OK) return rc;
  if (!aligned_to(n.xq, 16) || !aligned_to(n.q, 16) || !scales_aligned(n.scales, n.sfmt) ||
      !scales_aligned(n.x_scales, n.sfmt))
    return FP8_ERR_MISALIGNED;
  int sms = 0;
  if ((rc = sm_count(&sms)) != FP8_OK) return rc;
  fp8k::GatherArgs a{};
  a.x = codes ? n.xq : n.x;
  a.ldx = codes ? n.K : n.ld_x;
  a.x_scales = n.x_scales; a.rows = n.rows;
  a.T = n.T; a.S = n.S; a.K = n.K; a.M = n.M;
  a.fmt = n.fmt; a.sfmt = n.sfmt;
  a.q = n.q; a.scales = n.scales; a.out = n.out; a.ld_out = n.ld_out;
  const int source = codes ? fp8k::kGatherCodes
                           : n.dt == FP8_IN_BF16 ? fp8k::kGatherBf16 : fp8k::kGatherF32;
  return to_status(fp8k::launch_experts_gather(a, source, sms, (cudaStream_t)stream));
}

int fp8_experts_combine(const fp8_experts_combine_t *combine, fp8_stream_t stream) {
  const NvtxRange nvtx_range(__func__);
  if (combine == nullptr) return FP8_ERR_INVALID_ARG;
  const fp8_experts_combine_t &n = *combine;
  int rc = check_tokens(n.T, n.S, n.K, n.M, n.rows);
  if (rc == FP8_OK) rc = check_choices(n.S);
  if (rc != FP8_OK) return rc;
  if (!valid_in(n.x_dt) || !valid_in(n.out_dt)) return FP8_ERR_INVALID_ARG;
  if (n.T > 0 && (n.out == nullptr || (n.M > 0 && n.x == nullptr))) return FP8_ERR_INVALID_ARG;
  if ((rc = check_expert_rows(n.x, n.ld_x, n.K)) != FP8_OK) return rc;
  if ((rc = check_expert_rows(n.residual, n.ld_residual, n.K)) != FP8_OK) return rc;
  if ((rc = check_expert_rows(n.out, n.ld_out, n.K)) != FP8_OK) return rc;
  // in place each element is read before it is written, at the same place
  if (n.residual != nullptr && n.residual == n.out && n.ld_residual != n.ld_out)
    return FP8_ERR_INVALID_ARG;
  if (!aligned_to(n.weights, 4)) return FP8_ERR_MISALIGNED;
  int sms = 0;
  if ((rc = sm_count(&sms)) != FP8_OK) return rc;
  fp8k::CombineArgs a{};
  a.x = n.x; a.rows = n.rows; a.weights = n.weights; a.residual = n.residual; a.out = n.out;
  a.T = n.T; a.S = n.S; a.K = n.K; a.M = n.M;
  a.ldx = n.ld_x; a.ldr = n.ld_residual; a.ld_out = n.ld_out;
  return to_status(fp8k::launch_experts_combine(a, n.x_dt, n.out_dt, sms, (cudaStream_t)stream));
}

int fp8_experts_combine_backward(const fp8_experts_combine_grad_t *grad, fp8_stream_t stream) {
  const NvtxRange nvtx_range(__func__);
  if (grad == nullptr) return FP8_ERR_INVALID_ARG;
  const fp8_experts_combine_grad_t &n = *grad;
  int rc = check_tokens(n.T, n.S, n.K, n.M, n.rows);
  if (rc == FP8_OK) rc = check_choices(n.S);
  if (rc != FP8_OK) return rc;
  if (!valid_in(n.dy_dt) || !valid_in(n.x_dt) || !valid_in(n.dx_dt) || !valid_fmt(n.fmt) ||
      !valid_sfmt(n.sfmt))
    return FP8_ERR_INVALID_ARG;
  if ((n.q == nullptr) != (n.scales == nullptr)) return FP8_ERR_INVALID_ARG;
  if (n.T > 0) {
    if (n.dy == nullptr) return FP8_ERR_INVALID_ARG;
    if (n.d_weights != nullptr && n.M > 0 && n.x == nullptr) return FP8_ERR_INVALID_ARG;
    if (n.q == nullptr && n.dx == nullptr && n.d_weights == nullptr) return FP8_ERR_INVALID_ARG;
  }
  if ((rc = check_expert_rows(n.dy, n.ld_dy, n.K)) != FP8_OK) return rc;
  if ((rc = check_expert_rows(n.x, n.ld_x, n.K)) != FP8_OK) return rc;
  if ((rc = check_expert_rows(n.dx, n.ld_dx, n.K)) != FP8_OK) return rc;
  if (!aligned_to(n.weights, 4) || !aligned_to(n.d_weights, 4) || !aligned_to(n.q, 16) ||
      !scales_aligned(n.scales, n.sfmt))
    return FP8_ERR_MISALIGNED;
  int sms = 0;
  if ((rc = sm_count(&sms)) != FP8_OK) return rc;
  fp8k::CombineGradArgs a{};
  a.dy = n.dy; a.x = n.x; a.rows = n.rows; a.weights = n.weights; a.dw = n.d_weights;
  a.q = n.q; a.scales = n.scales; a.dx = n.dx;
  a.T = n.T; a.S = n.S; a.K = n.K; a.M = n.M;
  a.ld_dy = n.ld_dy; a.ldx = n.ld_x; a.ld_dx = n.ld_dx;
  a.fmt = n.fmt; a.sfmt = n.sfmt; a.dx_dt = n.dx_dt;
  return to_status(
      fp8k::launch_experts_combine_grad(a, n.dy_dt, n.x_dt, sms, (cudaStream_t)stream));
}

int fp8_act_checkpoint(const fp8_act_checkpoint_t *act, fp8_stream_t stream) {
  const NvtxRange nvtx_range(__func__);
  if (act == nullptr) return FP8_ERR_INVALID_ARG;
  const fp8_act_checkpoint_t &n = *act;
  if (n.M < 0 || n.N < 1 || n.M >= kMaxDim || n.N >= kMaxDim) return FP8_ERR_INVALID_ARG;
  if (n.act < FP8_ACT_NONE || n.act > FP8_ACT_GELU || !valid_fmt(n.fmt)) return FP8_ERR_INVALID_ARG;
  if (n.mode != FP8_NORM_TENSOR && n.mode != FP8_NORM_GROUP)
    return n.mode == FP8_NORM_MX ? FP8_ERR_UNSUPPORTED : FP8_ERR_INVALID_ARG;
  if (n.M > 0 && (n.h == nullptr || n.q == nullptr)) return FP8_ERR_INVALID_ARG;
  if (n.mode == FP8_NORM_TENSOR) {
    if (n.scale == nullptr || n.amax_out == n.scale || n.scales != nullptr) return FP8_ERR_INVALID_ARG;
  } else {
    if (!valid_sfmt(n.sfmt) || n.scale != nullptr) return FP8_ERR_INVALID_ARG;
    if (n.amax_out != nullptr) return FP8_ERR_UNSUPPORTED;
    if (n.M > 0 && n.scales == nullptr) return FP8_ERR_INVALID_ARG;
  }
  // both arguments are kept, or neither
  const bool keep = n.h_q != nullptr;
  if ((n.h_scales != nullptr) != keep || (n.u_q != nullptr) != (n.u_scales != nullptr) ||
      (n.M > 0 && (n.u_q != nullptr) != (keep && n.u != nullptr)) || (keep && !valid_sfmt(n.keep_sfmt)))
    return FP8_ERR_INVALID_ARG;
  if (n.N % 16 != 0) return FP8_ERR_MISALIGNED;
  int rc = check_rows(n.h, n.ld_h, n.N);
  if (rc == FP8_OK) rc = check_rows(n.u, n.ld_u, n.N);
  if (rc == FP8_OK) rc = check_rows(n.out, n.ld_out, n.N);
  if (rc != FP8_OK) return rc;
  if (!aligned_to(n.q, 16) || !aligned_to(n.h_q, 16) || !aligned_to(n.u_q, 16) ||
      !aligned_to(n.scale, 4) || !aligned_to(n.amax_out, 4) || !aligned_to(n.valid_rows, 4) ||
      !scales_aligned(n.scales, n.sfmt) || !scales_aligned(n.h_scales, n.keep_sfmt) ||
      !scales_aligned(n.u_scales, n.keep_sfmt))
    return FP8_ERR_MISALIGNED;
  int sms = 0;
  if ((rc = sm_count(&sms)) != FP8_OK) return rc;
  fp8k::ActArgs a{};
  a.h = n.h; a.u = n.u; a.M = n.M; a.N = n.N; a.ldh = n.ld_h; a.ldu = n.ld_u;
  a.valid = n.valid_rows; a.q = n.q; a.scale = n.scale; a.scales = n.scales;
  a.amax = reinterpret_cast<uint32_t *>(n.amax_out);
  a.hq = n.h_q; a.uq = n.u_q; a.hs = n.h_scales; a.us = n.u_scales;
  a.out = n.out; a.ld_out = n.ld_out;
  a.act = n.act; a.fmt = n.fmt; a.sfmt = n.sfmt; a.keep_sfmt = n.keep_sfmt;
  return to_status(fp8k::launch_act_checkpoint(a, sms, (cudaStream_t)stream));
}

int fp8_act_checkpoint_backward(const fp8_act_checkpoint_grad_t *grad, fp8_stream_t stream) {
  const NvtxRange nvtx_range(__func__);
  if (grad == nullptr) return FP8_ERR_INVALID_ARG;
  const fp8_act_checkpoint_grad_t &n = *grad;
  if (n.M < 0 || n.N < 1 || n.M >= kMaxDim || n.N >= kMaxDim) return FP8_ERR_INVALID_ARG;
  if (n.act < FP8_ACT_NONE || n.act > FP8_ACT_GELU || !valid_fmt(n.fmt) ||
      !valid_sfmt(n.keep_sfmt))
    return FP8_ERR_INVALID_ARG;
  if (n.mode != FP8_NORM_TENSOR && n.mode != FP8_NORM_GROUP)
    return n.mode == FP8_NORM_MX ? FP8_ERR_UNSUPPORTED : FP8_ERR_INVALID_ARG;
  if (n.M > 0 && (n.da == nullptr || n.h_q == nullptr || n.h_scales == nullptr))
    return FP8_ERR_INVALID_ARG;
  const bool gate = n.u_q != nullptr;
  if ((n.u_scales != nullptr) != gate) return FP8_ERR_INVALID_ARG;
  if (n.M > 0 && !gate && (n.du_q != nullptr || n.du != nullptr)) return FP8_ERR_INVALID_ARG;
  if (n.M > 0 && n.dh_q == nullptr && n.du_q == nullptr && n.dh == nullptr && n.du == nullptr)
    return FP8_ERR_INVALID_ARG;
  const float *sh = n.dh_q != nullptr ? n.scale_dh : nullptr;
  const float *su = n.du_q != nullptr ? n.scale_du : nullptr;
  if (n.mode == FP8_NORM_TENSOR) {
    if ((n.dh_q != nullptr && sh == nullptr) || (n.du_q != nullptr && su == nullptr))
      return FP8_ERR_INVALID_ARG;
    const float *am[2] = {n.amax_dh, n.amax_du};
    for (const float *p : am)
      if (p != nullptr && (p == n.scale_dh || p == n.scale_du)) return FP8_ERR_INVALID_ARG;
    if (n.amax_dh != nullptr && n.amax_dh == n.amax_du) return FP8_ERR_INVALID_ARG;
    if (n.M > 0 && ((n.amax_dh != nullptr && n.dh_q == nullptr) ||
                    (n.amax_du != nullptr && n.du_q == nullptr)))
      return FP8_ERR_UNSUPPORTED;  // a maximum without codes
  } else {
    if (!valid_sfmt(n.sfmt)) return FP8_ERR_INVALID_ARG;
    if (n.amax_dh != nullptr || n.amax_du != nullptr) return FP8_ERR_UNSUPPORTED;
    if ((n.dh_q != nullptr && n.dh_scales == nullptr) || (n.du_q != nullptr && n.du_scales == nullptr))
      return FP8_ERR_INVALID_ARG;
  }
  if (n.N % 16 != 0) return FP8_ERR_MISALIGNED;
  int rc = check_rows(n.da, n.ld_da, n.N);
  if (rc == FP8_OK) rc = check_rows(n.dh, n.ld_d, n.N);
  if (rc == FP8_OK) rc = check_rows(n.du, n.ld_d, n.N);
  if (rc != FP8_OK) return rc;
  if (n.dh_q != nullptr || n.du_q != nullptr) {
    if (n.ld_q < n.N || n.ld_q >= kMaxDim) return FP8_ERR_INVALID_ARG;
    if (n.ld_q % 16 != 0) return FP8_ERR_MISALIGNED;
  }
  if (!aligned_to(n.h_q, 16) || !aligned_to(n.u_q, 16) || !aligned_to(n.dh_q, 16) ||
      !aligned_to(n.du_q, 16) || !aligned_to(n.scale_dh, 4) || !aligned_to(n.scale_du, 4) ||
      !aligned_to(n.amax_dh, 4) || !aligned_to(n.amax_du, 4) || !aligned_to(n.valid_rows, 4) ||
      !scales_aligned(n.h_scales, n.keep_sfmt) || !scales_aligned(n.u_scales, n.keep_sfmt) ||
      !scales_aligned(n.dh_scales, n.sfmt) || !scales_aligned(n.du_scales, n.sfmt))
    return FP8_ERR_MISALIGNED;
  int sms = 0;
  if ((rc = sm_count(&sms)) != FP8_OK) return rc;
  const bool tensor = n.mode == FP8_NORM_TENSOR;
  fp8k::ActGradArgs a{};
  a.da = n.da; a.ld_da = n.ld_da; a.hq = n.h_q; a.uq = n.u_q; a.hs = n.h_scales; a.us = n.u_scales;
  a.M = n.M; a.N = n.N; a.valid = n.valid_rows;
  a.qh = n.dh_q; a.qu = n.du_q; a.ld_q = n.ld_q;
  a.tensor = tensor ? 1 : 0;
  a.scale_h = tensor ? sh : nullptr;
  a.scale_u = tensor ? su : nullptr;
  a.sh = n.dh_scales; a.su = n.du_scales;
  a.amax_h = reinterpret_cast<uint32_t *>(n.amax_dh);
  a.amax_u = reinterpret_cast<uint32_t *>(n.amax_du);
  a.dh = n.dh; a.du = n.du; a.ld_d = n.ld_d;
  a.act = n.act; a.fmt = n.fmt; a.sfmt = n.sfmt; a.keep_sfmt = n.keep_sfmt;
  return to_status(fp8k::launch_act_checkpoint_grad(a, sms, (cudaStream_t)stream));
}

}  // extern "C"
