// launch.cuh -- host side of launches: a kernel's shared-memory opt-in, the code
// of a launch with attributes.
#pragma once

#include "common.cuh"

namespace flide {

// Lets `kKernel` take all the dynamic shared memory an SM gives one block, once
// per device (the first 64 are remembered).
template <auto kKernel>
bool allow_smem(int dev) {
  static std::atomic<bool> done[64];  // zero-initialised: false
  if (dev >= 0 && dev < 64 && done[dev].load(std::memory_order_acquire)) return true;
  cudaFuncAttributes at;
  int most = 0;
  if (cudaFuncGetAttributes(&at, kKernel) != cudaSuccess ||
      cudaDeviceGetAttribute(&most, cudaDevAttrMaxSharedMemoryPerBlockOptin, dev) != cudaSuccess ||
      cudaFuncSetAttribute(kKernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           most - (int)at.sharedSizeBytes) != cudaSuccess)
    return false;
  if (dev >= 0 && dev < 64) done[dev].store(true, std::memory_order_release);
  return true;
}

// The code of a cudaLaunchKernelEx; its error does not stay behind for the next call.
inline int launched(cudaError_t e) {
  if (e == cudaSuccess) return FLIDE_OK;
  cudaGetLastError();
  return FLIDE_ERR_CUDA;
}

}  // namespace flide
