// Dynamic shared memory of a kernel, asked for once per device and size (the
// attribute call costs the host 0.3 us, which single-token calls notice).
#pragma once

#include <cuda_runtime_api.h>

#include <atomic>
#include <mutex>

namespace fattn {

class SmemLimit {
 public:
  // After success the kernel may be launched with `bytes` on the current
  // device, whatever other threads ask for: the limit is set by one thread at a
  // time and never lowered, so that none falls between another's request and
  // its launch.
  cudaError_t raise(const void* kernel, int bytes) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= kDevices) return cudaErrorInvalidDevice;
    if (bytes_[dev].load(std::memory_order_acquire) >= bytes) return cudaSuccess;
    std::lock_guard<std::mutex> lock(mu_);
    if (bytes_[dev].load(std::memory_order_relaxed) >= bytes) return cudaSuccess;
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == cudaSuccess) bytes_[dev].store(bytes, std::memory_order_release);
    return e;
  }

 private:
  static constexpr int kDevices = 64;
  std::mutex mu_;
  std::atomic<int> bytes_[kDevices] = {};
};

}  // namespace fattn
