// Launches with programmatic stream serialization: the kernel may start before
// the previous one in the stream ends, and waits for it (grid_dependency_wait)
// before it touches memory.  What the previous kernel writes is not constant
// over such a kernel's lifetime: it is read with plain loads, never through the
// read-only path (__ldg, const __restrict__).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>

namespace fp8k {

// `cluster` CTAs of a thread-block cluster (1: none); blocks is a multiple.
template <typename... KArgs, typename... Args>
cudaError_t launch_serial_cluster(void (*kern)(KArgs...), int64_t blocks, int threads, int cluster,
                                  int smem, cudaStream_t st, Args... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.dynamicSmemBytes = (size_t)smem;
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
  return launch_serial_cluster(kern, blocks, threads, 1, 0, st, args...);
}

// Sets an attribute of a kernel once per device.
template <auto KERN, cudaFuncAttribute ATTR>
cudaError_t allow_once(int value) {
  static std::atomic<uint64_t> allowed{0};  // a bit per device
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = (uint64_t)1 << (dev & 63);
  if ((allowed.load(std::memory_order_relaxed) & bit) == 0) {
    e = cudaFuncSetAttribute(KERN, ATTR, value);
    if (e != cudaSuccess) return e;
    allowed.fetch_or(bit, std::memory_order_relaxed);
  }
  return cudaSuccess;
}

// With dynamic shared memory that may exceed 48 KB (at most MOST).
template <auto KERN, int MOST, typename... Args>
cudaError_t launch_serial_smem(int64_t blocks, int threads, int smem, cudaStream_t st,
                               Args... args) {
  const cudaError_t e = allow_once<KERN, cudaFuncAttributeMaxDynamicSharedMemorySize>(MOST);
  if (e != cudaSuccess) return e;
  return launch_serial_cluster(KERN, blocks, threads, 1, smem, st, args...);
}

// `most` (more than eight) where the device can hold a cluster of that many of
// this kernel's CTAs, else eight; asked once per device.
template <auto KERN>
int widest_cluster(int most, int threads) {
  static std::atomic<uint64_t> asked{0}, wide{0};  // a bit per device
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 8;
  const uint64_t bit = (uint64_t)1 << (dev & 63);
  if ((asked.load(std::memory_order_acquire) & bit) == 0) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)most);
    cfg.blockDim = dim3((unsigned)threads);
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)most;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    int held = 0;
    if (cudaFuncSetAttribute(KERN, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) == cudaSuccess &&
        cudaOccupancyMaxActiveClusters(&held, KERN, &cfg) == cudaSuccess && held > 0)
      wide.fetch_or(bit, std::memory_order_relaxed);
    else
      (void)cudaGetLastError();
    asked.fetch_or(bit, std::memory_order_release);
  }
  return wide.load(std::memory_order_relaxed) & bit ? most : 8;
}

}  // namespace fp8k
