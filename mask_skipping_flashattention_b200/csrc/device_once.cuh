// A kernel's attributes are set once on every device it runs on (they belong to the
// device's context, not to the process).
#pragma once

#include <atomic>
#include <cuda_runtime.h>

namespace bfa {

struct DeviceOnce {
  static constexpr int kMaxDevices = 64;
  std::atomic<bool> done[kMaxDevices] = {};
  template <typename F>
  cudaError_t run(F&& f) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
    if (done[dev].load(std::memory_order_acquire)) return cudaSuccess;
    e = f();  // two threads may both do it: the same values twice
    if (e == cudaSuccess) done[dev].store(true, std::memory_order_release);
    return e;
  }
};

}  // namespace bfa
