// Launchers of the kernels that take tokens to their experts' rows and back
// (experts.cu).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace fp8k {

// Stable order of P (token, choice) pairs by expert: offsets [E + 1], the row
// of each pair (-1: its id is outside [0, E)), and (nullable) the pair of each
// row, -1 behind the last.
cudaError_t launch_experts_sort(const void *ids, bool wide, int64_t P, int E, int32_t *offsets,
                                int32_t *rows, int32_t *pairs, cudaStream_t st);

// Pair (t, s) is row rows[t * S + s] of the [M, K] side; rows outside [0, M)
// are dropped pairs.
struct GatherArgs {
  const void *x;          // [T, ldx] bf16 or fp32, or codes [T, K]
  const void *x_scales;   // codes only: [ceil(K/128), T]
  const int32_t *rows;
  int64_t T, S, K, M, ldx;
  int fmt, sfmt;
  uint8_t *q;             // nullable (with out): [M, K]
  void *scales;           // [ceil(K/128), M]
  void *out;              // nullable: rows of x's type
  int64_t ld_out;
};
enum GatherSource : int { kGatherBf16 = 0, kGatherF32 = 1, kGatherCodes = 2 };
cudaError_t launch_experts_gather(const GatherArgs &a, int source, int sms, cudaStream_t st);

struct CombineArgs {
  const void *x;          // [M, ldx]
  const int32_t *rows;
  const float *weights;   // nullable [T, S]: ones
  const void *residual;   // nullable [T, ldr] of the output's type
  void *out;              // [T, ld_out]
  int64_t T, S, K, M, ldx, ldr, ld_out;
};
cudaError_t launch_experts_combine(const CombineArgs &a, int x_dt, int out_dt, int sms,
                                   cudaStream_t st);

struct CombineGradArgs {
  const void *dy;         // [T, ld_dy]
  const void *x;          // nullable (no dw): [M, ldx]
  const int32_t *rows;
  const float *weights;   // nullable: ones
  float *dw;              // nullable [T, S]
  uint8_t *q;             // nullable [M, K]
  void *scales;           // with q: [ceil(K/128), M]
  void *dx;               // nullable [M, ld_dx]
  int64_t T, S, K, M, ld_dy, ldx, ld_dx;
  int fmt, sfmt, dx_dt;
  int alone;              // a warp takes a token alone (set by the launcher)
};
cudaError_t launch_experts_combine_grad(const CombineGradArgs &a, int dy_dt, int x_dt, int sms,
                                        cudaStream_t st);

}  // namespace fp8k
