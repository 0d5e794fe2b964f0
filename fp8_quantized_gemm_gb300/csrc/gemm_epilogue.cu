// The general GEMM kernel (gemm_kernel.cuh) with the linear layer's epilogue:
// the shapes the CTA-pair and few-row kernels do not take.
#include "gemm_kernel.cuh"

namespace fp8k {

cudaError_t launch_gemm_epilogue(int mode, const CUtensorMap &tma, const CUtensorMap &tmb,
                                 const GemmArgs &args, const LinearEp &ep, int sms,
                                 cudaStream_t st) {
  const EpParam<true> p{ep};
  const bool mc = args.multicast != 0;
  switch (mode) {
    case kScaleTensor:
      if (mc) return cudaErrorInvalidValue;
      return run<kScaleTensor, 256, 4, false, 1, true>(tma, tmb, args, sms, st, p);
    case kScaleMx:
      if (gemm_tile_n(mode, args.M, args.N, sms) != 128)
        return mc ? cudaErrorInvalidValue
                  : run<kScaleMx, 256, 4, false, 1, true>(tma, tmb, args, sms, st, p);
      return mc ? run<kScaleMx, 128, 6, false, 2, true>(tma, tmb, args, sms, st, p)
                : run<kScaleMx, 128, 6, false, 1, true>(tma, tmb, args, sms, st, p);
    case kScaleGroupF32:
      return mc ? run<kScaleGroupF32, 128, kF32Stages, false, 2, true>(tma, tmb, args, sms, st, p)
                : run<kScaleGroupF32, 128, kF32Stages, false, 1, true>(tma, tmb, args, sms, st, p);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace fp8k
