// The limit of a kernel's dynamic shared memory.  It is 48 KB until it is raised,
// and a raise holds for one device: every launch of more asks here first, so
// that a process may use the kernels on several devices.
#pragma once
#include <cuda_runtime_api.h>

#include <map>
#include <mutex>
#include <utility>

namespace mlpk {

// Lets `func` be launched with `bytes` of dynamic shared memory on the current
// device.  Raised once per device, kernel and size; a failure is returned and
// the next launch tries again.
inline cudaError_t allow_smem(const void* func, unsigned bytes) {
  if (bytes <= 48u * 1024u) return cudaSuccess;
  int device = 0;
  cudaError_t e = cudaGetDevice(&device);
  if (e != cudaSuccess) return e;
  static std::mutex mu;
  static std::map<std::pair<int, const void*>, unsigned> allowed;
  try {
    std::lock_guard<std::mutex> lock(mu);
    unsigned& have = allowed[{device, func}];
    if (have >= bytes) return cudaSuccess;
    e = cudaFuncSetAttribute(func, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
    if (e == cudaSuccess) have = bytes;
    return e;
  } catch (...) {   // (no exception leaves a C entry)
    return cudaErrorMemoryAllocation;
  }
}

}  // namespace mlpk
