// The general GEMM kernel (gemm_kernel.cuh) with the linear layer's epilogue:
// the shapes the CTA-pair and few-row kernels do not take.
#include "gemm_kernel.cuh"

namespace fp8k {

// Per-tensor scales: 128-wide tiles (the kernel runs here with fewer output
// tiles than the CTA pairs need; narrow ones occupy more SMs and leave each
// warp half the epilogue).  Block-scale words: where the plain kernel takes
// 256-wide tiles (one TMEM accumulator beside the scale factors: the epilogue
// of a tile and the MMAs of the next take turns), 192-wide ones, two of which
// fit: 4096 x 7168 x 2048 with bias and silu runs in 54.2 us, B multicast to
// the two CTAs of a cluster (2-3 us more without), against 72.1 on 256-wide
// tiles.  With few columns and a deep K (4096 x 2048 x 7168) the two are near:
// 57.2 against 59.9.
int gemm_epilogue_tile_n(int mode, int64_t M, int64_t N, int sms) {
  const int bn = gemm_tile_n(mode, M, N, sms);
  if (mode == kScaleTensor) return 128;
  return mode == kScaleMx && bn == 256 ? 192 : bn;
}

cudaError_t launch_gemm_epilogue(int mode, const CUtensorMap &tma, const CUtensorMap &tmb,
                                 const GemmArgs &args, const LinearEp &ep, bool grad, int sms,
                                 cudaStream_t st) {
  const EpParam<true> p{ep};
  const bool mc = args.multicast != 0;
  if (grad && (mode != kScaleTensor || args.ksplit != 1)) return cudaErrorInvalidValue;
  switch (mode) {
    case kScaleTensor:
      if (mc) return cudaErrorInvalidValue;
      return grad ? run<kScaleTensor, 128, 5, false, 1, 2>(tma, tmb, args, sms, st, p)
                  : run<kScaleTensor, 128, 5, false, 1, 1>(tma, tmb, args, sms, st, p);
    case kScaleMx:
      if (gemm_epilogue_tile_n(mode, args.M, args.N, sms) == 192)
        return mc ? run<kScaleMx, 192, 4, false, 2, 1>(tma, tmb, args, sms, st, p)
                  : run<kScaleMx, 192, 4, false, 1, 1>(tma, tmb, args, sms, st, p);
      return mc ? run<kScaleMx, 128, 5, false, 2, 1>(tma, tmb, args, sms, st, p)
                : run<kScaleMx, 128, 5, false, 1, 1>(tma, tmb, args, sms, st, p);
    case kScaleGroupF32:
      return mc ? run<kScaleGroupF32, 128, kF32Stages, false, 2, 1>(tma, tmb, args, sms, st, p)
                : run<kScaleGroupF32, 128, kF32Stages, false, 1, 1>(tma, tmb, args, sms, st, p);
    default: return cudaErrorInvalidValue;
  }
}

// Clusters of `size` CTAs of the 128-wide per-tensor kernel resident at once.
static int clusters_cached(int size) {
  static int cache[64][kMaxClusterSplit + 1];
  static bool have[64][kMaxClusterSplit + 1];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 0;
  if (!have[dev][size]) {
    cache[dev][size] = active_clusters<kScaleTensor, 128, 5, 1, 1>(size);
    have[dev][size] = true;
  }
  return cache[dev][size];
}

// K splits of a per-tensor problem on 128-wide tiles (gemm_ksplit's rule).
int gemm_epilogue_ksplit(int64_t M, int64_t N, int64_t K, int sms) {
  const int64_t tiles = (M + 127) / 128 * ((N + 127) / 128), kb = (K + 127) / 128;
  if (tiles * 2 > sms || kb < 8) return 1;
  int64_t ks = sms / tiles;
  if (ks > kb / 4) ks = kb / 4;
  if (ks > kMaxClusterSplit) ks = kMaxClusterSplit;
  while (ks > 1 && clusters_cached((int)ks) < tiles) --ks;
  return ks < 2 ? 1 : (int)ks;
}

}  // namespace fp8k
