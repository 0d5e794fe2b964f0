// Device scratch of calls that take none from their caller (workspace.cu).
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>

#include <mutex>

namespace fp8k {

// Not initialised, for the kernels that the calling thread enqueues on `st`
// while the object lives.  Successive ones on a stream share memory, so an
// object holds off the other threads' until it is gone (they may enqueue on the
// same stream).
class Workspace {
 public:
  Workspace() = default;
  ~Workspace();
  Workspace(const Workspace &) = delete;
  Workspace &operator=(const Workspace &) = delete;
  cudaError_t get(cudaStream_t st, size_t need);  // once per object
  void *ptr() const { return ptr_; }

 private:
  cudaError_t find(cudaStream_t st, size_t need);

  std::unique_lock<std::mutex> lock_;
  void *ptr_ = nullptr;
  cudaStream_t st_ = nullptr;
  bool ordered_ = false;  // allocated in the stream's order: freed in it too
};

}  // namespace fp8k
