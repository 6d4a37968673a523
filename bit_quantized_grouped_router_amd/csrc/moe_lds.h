// More than 64 KB of dynamic LDS needs an opt-in for each kernel and device.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <atomic>

namespace moe {

// `done` is the kernel's own: a bit for each device that has been asked.
inline hipError_t allow_lds(const void *kernel, int bytes, std::atomic<uint64_t> &done) {
  int device = 0;
  const hipError_t e = hipGetDevice(&device);
  if (e != hipSuccess) return e;
  const uint64_t bit = device < 64 ? 1ull << device : 0;
  if (done.load(std::memory_order_relaxed) & bit) return hipSuccess;
  const hipError_t st = hipFuncSetAttribute(kernel, hipFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (st == hipSuccess) done.fetch_or(bit, std::memory_order_relaxed);
  return st;
}

}  // namespace moe
