// Launchers of the RMS norm kernels (norm.cu) and of the column sums that
// finish dw and dbias.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace fp8k {

enum NormMode : int { kNormTensor = 0, kNormGroup = 1, kNormMx = 2 };

constexpr int64_t kNormMaxK = 16384;  // two vectors of 8 for each of 1024 threads

struct NormArgs {
  const void *x, *res, *w;  // res, w nullable
  void *sum, *y;            // nullable
  uint8_t *q;
  const float *scale;       // kNormTensor
  void *scales;             // kNormGroup: [ceil(K/128), M]; kNormMx: words [K/128][M padded]
  float *inv_rms;           // nullable [M]
  uint32_t *amax;           // nullable (kNormTensor)
  int64_t M, K, ldx, ldr, ld_sum, ld_y;
  float eps, inv_k;         // inv_k = 1 / K
  int fmt, sfmt, w_dt;
};
cudaError_t launch_rmsnorm(const NormArgs &a, int dt, int mode, int sms, cudaStream_t st);

struct NormGradArgs {
  const void *dy, *r, *w, *dres;  // w, dres nullable
  const float *inv_rms;
  void *dx;
  float *parts;                   // nullable: dw partials [blocks][K]
  uint32_t *tops;                 // nullable, with parts and amax: max |dx| of each CTA
  uint8_t *q;                     // nullable
  const float *scale;
  uint32_t *amax;                 // nullable
  int64_t M, K, ld_dy, ld_r, ld_dres, ld_dx;
  float inv_k;
  int fmt, w_dt;
};
// Rows of partial sums the backward pass writes for dw on a device of `sms`
// multiprocessors.
int64_t rmsnorm_grad_blocks(int64_t M, int64_t K, int sms);
cudaError_t launch_rmsnorm_grad(const NormGradArgs &a, int dt, int dy_dt, float *dw,
                                int accumulate, int sms, cudaStream_t st);

// out[n] (+)= sum over p < P of parts[p][n]; *top_out (nullable) = max of tops
cudaError_t launch_column_sum(const float *parts, int64_t P, int64_t N, int accumulate, float *out,
                              const float *tops, int ntops, uint32_t *top_out, cudaStream_t st);
// *p = 0, in the programmatic launch chain
cudaError_t launch_clear_word(uint32_t *p, cudaStream_t st);

}  // namespace fp8k
