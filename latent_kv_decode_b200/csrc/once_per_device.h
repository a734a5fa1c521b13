// A kernel attribute set once per device instead of once per launch (internal).
#pragma once

#include <cuda_runtime.h>

#include <atomic>

namespace mla {

// Bits of the devices for which `set` has succeeded.
class OncePerDevice {
 public:
  // Run set() unless it has succeeded on the current device (numbers 0-63;
  // others run it every time). Threads may run it at the same time: setting an
  // attribute twice to the same value is harmless.
  template <typename F>
  cudaError_t operator()(F set) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const unsigned long long bit = dev >= 0 && dev < 64 ? 1ull << dev : 0ull;
    if (done_.load(std::memory_order_acquire) & bit) return cudaSuccess;
    e = set();
    if (e == cudaSuccess) done_.fetch_or(bit, std::memory_order_release);
    return e;
  }

 private:
  std::atomic<unsigned long long> done_{0};
};

}  // namespace mla
