// Launches of the general GEMM kernel (gemm_kernel.cuh): tile widths, K
// splits and the variants of each scale mode.
#include "gemm_kernel.cuh"

namespace fp8k {

// Tile width: 128 for the FP32-promotion mode; 256 for the per-tensor mode
// (whose large shapes run on CTA pairs); for the block-scaled modes 256 when
// the 128 x 256 tiles fill the SMs and 128 otherwise (twice the tiles: mid-
// size M then needs no split K, small M splits K over fewer k blocks).
int gemm_tile_n(int mode, int64_t M, int64_t N, int sms) {
  if (mode == kScaleGroupF32 || mode == kScaleGroupF32x32) return 128;
  if (mode == kScaleTensor) return 256;
  const int64_t tiles256 = ((M + 127) / 128) * ((N + 255) / 256);
  return tiles256 < sms ? 128 : 256;
}

// Split K when the tiles cannot fill half the SMs: as many splits as fit the
// SMs, each covering at least four 128-wide K blocks.  Cluster splits reduce
// through distributed shared memory (at most kMaxClusterSplit per tile);
// workspace splits are capped at 512 KB of fp32 partials per tile, which the
// last CTA of the tile sums.
static int max_active_clusters(int mode, int bn, int size) {
  static int cache[64][5][2][kMaxClusterSplit + 1];
  static bool have[64][5][2][kMaxClusterSplit + 1];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 0;
  const int w = bn == 128 ? 0 : 1;
  if (!have[dev][mode][w][size]) {
    int n = 0;
    switch (mode) {
      case kScaleTensor: n = active_clusters<kScaleTensor, 256, 4>(size); break;
      case kScaleMx:
        n = w == 0 ? active_clusters<kScaleMx, 128, 6>(size)
                   : active_clusters<kScaleMx, 256, 4>(size);
        break;
      case kScaleGroupUe8m0:
        n = w == 0 ? active_clusters<kScaleGroupUe8m0, 128, 6>(size)
                   : active_clusters<kScaleGroupUe8m0, 256, 4>(size);
        break;
      case kScaleGroupF32x32: n = active_clusters<kScaleGroupF32x32, 128, kF32Stages>(size); break;
      default: n = active_clusters<kScaleGroupF32, 128, kF32Stages>(size); break;
    }
    cache[dev][mode][w][size] = n;
    have[dev][mode][w][size] = true;
  }
  return cache[dev][mode][w][size];
}

int gemm_ksplit(int mode, int64_t M, int64_t N, int64_t K, int sms, bool cluster) {
  const int64_t bn = gemm_tile_n(mode, M, N, sms);
  const int64_t tiles = ((M + 127) / 128) * ((N + bn - 1) / bn);
  const int64_t kb = (K + 127) / 128;
  if (tiles * 2 > sms || kb < 8) return 1;
  int64_t ks = sms / tiles;
  if (ks > kb / 4) ks = kb / 4;
  if (cluster) {
    // the largest split whose clusters (one per tile) are all resident at
    // once: a second wave of clusters would double the time
    if (ks > kMaxClusterSplit) ks = kMaxClusterSplit;
    while (ks > 1 && max_active_clusters(mode, (int)bn, (int)ks) < tiles) --ks;
  } else {
    const int64_t rows = M < 128 ? M : 128;
    const int64_t by_partials = (512 * 1024) / (rows * bn * 4);
    if (ks > by_partials) ks = by_partials;
  }
  return ks < 2 ? 1 : (int)ks;
}

cudaError_t launch_gemm_experts(int mode, int bn, const CUtensorMap &tma, const CUtensorMap &tmb,
                                const GemmArgs &args, int sms, cudaStream_t st) {
  // (six stages: the expert tables take 3 KB of static shared memory)
  if (mode == kScaleGroupF32) return run<kScaleGroupF32, 128, 6, true>(tma, tmb, args, sms, st);
  if (mode == kScaleMx) {
    if (bn == 128) return run<kScaleMx, 128, 6, true>(tma, tmb, args, sms, st);
    return run<kScaleMx, 256, 4, true>(tma, tmb, args, sms, st);
  }
  if (mode != kScaleGroupUe8m0) return cudaErrorInvalidValue;
  if (bn == 128) return run<kScaleGroupUe8m0, 128, 6, true>(tma, tmb, args, sms, st);
  return run<kScaleGroupUe8m0, 256, 4, true>(tma, tmb, args, sms, st);
}

cudaError_t launch_gemm(int mode, const CUtensorMap &tma, const CUtensorMap &tmb,
                        const GemmArgs &args, int sms, cudaStream_t st) {
  const bool mc = args.multicast != 0;
  if (mc && mode == kScaleTensor) return cudaErrorInvalidValue;
  switch (mode) {
    case kScaleTensor: return run<kScaleTensor, 256, 4>(tma, tmb, args, sms, st);
    case kScaleMx:
      if (gemm_tile_n(mode, args.M, args.N, sms) == 128)
        return mc ? run<kScaleMx, 128, 6, false, 2>(tma, tmb, args, sms, st)
                  : run<kScaleMx, 128, 6>(tma, tmb, args, sms, st);
      return mc ? run<kScaleMx, 256, 4, false, 2>(tma, tmb, args, sms, st)
                : run<kScaleMx, 256, 4>(tma, tmb, args, sms, st);
    case kScaleGroupUe8m0:
      if (gemm_tile_n(mode, args.M, args.N, sms) == 128)
        return mc ? run<kScaleGroupUe8m0, 128, 6, false, 2>(tma, tmb, args, sms, st)
                  : run<kScaleGroupUe8m0, 128, 6>(tma, tmb, args, sms, st);
      return mc ? run<kScaleGroupUe8m0, 256, 4, false, 2>(tma, tmb, args, sms, st)
                : run<kScaleGroupUe8m0, 256, 4>(tma, tmb, args, sms, st);
    case kScaleGroupF32:
      return mc ? run<kScaleGroupF32, 128, kF32Stages, false, 2>(tma, tmb, args, sms, st)
                : run<kScaleGroupF32, 128, kF32Stages>(tma, tmb, args, sms, st);
    case kScaleGroupF32x32:
      if (mc) return cudaErrorInvalidValue;
      return run<kScaleGroupF32x32, 128, kF32Stages>(tma, tmb, args, sms, st);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace fp8k
