// Dynamic shared memory of a kernel: the driver's limit, raised where a launch needs more.
#pragma once

#include <cuda_runtime_api.h>

#include <atomic>
#include <mutex>

#include "../../include/moe_verify.h"

namespace moe {

// Lets kernel K use `bytes` of dynamic shared memory; asks the driver once per device and size.  One thread at a time
// does, and only for more: a smaller request after a larger one would take the larger one's limit back.
template <auto K>
int allow_smem(size_t bytes) {
  static std::atomic<size_t> allowed[64];
  static std::mutex mu;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return MOE_ERR_CUDA;
  const bool noted = dev >= 0 && dev < 64;
  if (noted && allowed[dev].load(std::memory_order_acquire) >= bytes) return MOE_OK;
  std::lock_guard<std::mutex> lk(mu);
  if (noted && allowed[dev].load(std::memory_order_relaxed) >= bytes) return MOE_OK;
  if (cudaFuncSetAttribute(reinterpret_cast<const void*>(K), cudaFuncAttributeMaxDynamicSharedMemorySize,
                           static_cast<int>(bytes)) != cudaSuccess)
    return MOE_ERR_CUDA;
  if (noted) allowed[dev].store(bytes, std::memory_order_release);
  return MOE_OK;
}

}  // namespace moe
