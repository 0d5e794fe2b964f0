// Launches with programmatic stream serialization: the kernel may start before
// the previous one in the stream ends, and waits for it (grid_dependency_wait)
// before it touches memory.  What the previous kernel writes is not constant
// over such a kernel's lifetime: it is read with plain loads, never through the
// read-only path (__ldg, const __restrict__).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace fp8k {

// `cluster` CTAs of a thread-block cluster (1: none); blocks is a multiple.
template <typename... KArgs, typename... Args>
cudaError_t launch_serial_cluster(void (*kern)(KArgs...), int64_t blocks, int threads, int cluster,
                                  cudaStream_t st, Args... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)blocks);
  cfg.blockDim = dim3((unsigned)threads);
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = (unsigned)cluster;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kern, args...);
}

template <typename... KArgs, typename... Args>
cudaError_t launch_serial(void (*kern)(KArgs...), int64_t blocks, int threads, cudaStream_t st,
                          Args... args) {
  return launch_serial_cluster(kern, blocks, threads, 1, st, args...);
}

}  // namespace fp8k
