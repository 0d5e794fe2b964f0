// Launchers of the activation that keeps its arguments in 8 bits for the
// backward pass (act_checkpoint.cu).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace fp8k {

// A checkpoint: E4M3 codes [M, N] with a scale per 1x128 group, [ceil(N/128), M].
struct ActArgs {
  const void *h, *u;          // bf16 [M, ld]; u nullable (no gate)
  int64_t M, N, ldh, ldu;
  const int32_t *valid;       // nullable: rows at and behind valid[0] are left alone
  uint8_t *q;                 // codes of a [M, N]
  const float *scale;         // per tensor, or
  void *scales;               // per 1x128 group (scale null)
  uint32_t *amax;             // nullable, per tensor
  uint8_t *hq, *uq;           // nullable checkpoints
  void *hs, *us;
  void *out;                  // nullable bf16 a [M, ld_out]
  int64_t ld_out;
  int act, fmt, sfmt, keep_sfmt;
};
cudaError_t launch_act_checkpoint(const ActArgs &a, int sms, cudaStream_t st);

struct ActGradArgs {
  const void *da;             // bf16 [M, ld_da]
  const uint8_t *hq, *uq;     // checkpoints; uq nullable (no gate)
  const void *hs, *us;
  int64_t M, N, ld_da;
  const int32_t *valid;
  uint8_t *qh, *qu;           // nullable codes of dh, du [M, ld_q]
  int64_t ld_q;
  int tensor;                      // 1: codes under scale_h and scale_u
  const float *scale_h, *scale_u;
  void *sh, *su;                   // 0: scales per 1x128 group
  uint32_t *amax_h, *amax_u;       // nullable, per tensor
  void *dh, *du;              // nullable bf16 [M, ld_d]
  int64_t ld_d;
  int act, fmt, sfmt, keep_sfmt;
};
cudaError_t launch_act_checkpoint_grad(const ActGradArgs &a, int sms, cudaStream_t st);

}  // namespace fp8k
