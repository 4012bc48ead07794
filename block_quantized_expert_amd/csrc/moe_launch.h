// What launches of kernels with much LDS share.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <atomic>

namespace moe {

// Kernels that ask for more than 64 KB of dynamic LDS say so, at most `Bytes`,
// once for each device that they are launched on: the permission is the
// current device's, not the process's.
template <auto Kernel, int Bytes>
hipError_t allow_lds() {
  static std::atomic<uint64_t> allowed{0};  // of devices 0 to 63; others say so each time
  int device = 0;
  hipError_t e = hipGetDevice(&device);
  if (e != hipSuccess) return e;
  const uint64_t bit = device < 64 ? uint64_t{1} << device : 0;
  if ((allowed.load(std::memory_order_relaxed) & bit) != 0) return hipSuccess;
  e = hipFuncSetAttribute(reinterpret_cast<const void*>(Kernel),
                          hipFuncAttributeMaxDynamicSharedMemorySize, Bytes);
  if (e == hipSuccess) allowed.fetch_or(bit, std::memory_order_relaxed);
  return e;
}

}  // namespace moe
