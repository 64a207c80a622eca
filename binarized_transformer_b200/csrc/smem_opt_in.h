// smem_opt_in.h -- the dynamic shared-memory opt-in of a kernel (host code).
#pragma once

#include <atomic>
#include <mutex>

#include <cuda_runtime_api.h>

namespace bwta {

// The >48 KB dynamic shared-memory opt-in of one kernel, made once per device
// (the device current at the call) and again for a larger size. Only a success is
// remembered, so a call that failed is retried on the next launch. Host threads may
// call at once: the attribute and the record of it change together, so a smaller
// size never replaces a larger one that a launch counts on. With max_carveout the
// kernel also asks for the largest shared-memory carveout, so that an SM running one
// of its CTAs keeps room for a CTA of the next kernel in the stream (left to itself
// the driver may size the carveout for this kernel's CTA alone).
class SmemOptIn {
 public:
  template <typename Kern>
  cudaError_t operator()(Kern *kern, int bytes, bool max_carveout = false) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const bool cached = dev >= 0 && dev < kDevices;
    if (cached && set_[dev].load(std::memory_order_acquire) >= bytes) return cudaSuccess;
    std::lock_guard<std::mutex> lock(mutex_);
    if (cached && set_[dev].load(std::memory_order_relaxed) >= bytes) return cudaSuccess;
    const void *fn = reinterpret_cast<const void *>(kern);
    e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == cudaSuccess && max_carveout)
      e = cudaFuncSetAttribute(fn, cudaFuncAttributePreferredSharedMemoryCarveout,
                               (int)cudaSharedmemCarveoutMaxShared);
    if (e == cudaSuccess && cached) set_[dev].store(bytes, std::memory_order_release);
    return e;
  }

 private:
  static constexpr int kDevices = 64;
  std::atomic<int> set_[kDevices] = {};
  std::mutex mutex_;
};

}  // namespace bwta
