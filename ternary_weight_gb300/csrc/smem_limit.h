// smem_limit.h -- a kernel's dynamic shared memory limit (and leave for clusters of more than 8 blocks), set once on each device.
#pragma once

#include <atomic>
#include <cstdint>

#include <cuda_runtime.h>

namespace bitnet {

// `configured`: a static of the caller's, one for each kernel (a bit a device; the calls are allowed on 64).
template <typename Kernel>
cudaError_t allow_smem(std::atomic<uint64_t>& configured, Kernel kernel, int bytes, bool wide_clusters = false) {
  int dev = 0;
  if (cudaError_t e = cudaGetDevice(&dev)) return e;
  const uint64_t bit = 1ull << (dev & 63);
  if (configured.load(std::memory_order_acquire) & bit) return cudaSuccess;
  if (cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes)) return e;
  if (wide_clusters)
    if (cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1)) return e;
  configured.fetch_or(bit, std::memory_order_acq_rel);
  return cudaSuccess;
}

}  // namespace bitnet
