// Host helpers of the C ABI translation units: argument checks and the device's SM count.
#pragma once

#include <atomic>
#include <initializer_list>

#include "common.cuh"

namespace moe {

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// All listed pointers must be non-null and 16-byte aligned.
inline moe_status check_ptrs(std::initializer_list<const void*> ps) {
  for (const void* p : ps)
    if (!p || !aligned16(p)) return MOE_ERR_INVALID_ARG;
  return MOE_OK;
}

inline int num_sms() {
  static std::atomic<int> cached[64];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 148;
  int n = cached[dev].load(std::memory_order_relaxed);
  if (!n) {
    int v = 0;
    cudaDeviceGetAttribute(&v, cudaDevAttrMultiProcessorCount, dev);
    n = v > 0 ? v : 148;
    cached[dev].store(n, std::memory_order_relaxed);
  }
  return n;
}

moe_status check_route(const moe_route_desc* d);

#define MOE_TRY(expr)                 \
  do {                                \
    moe_status _s = (expr);           \
    if (_s != MOE_OK) return _s;      \
  } while (0)

}  // namespace moe
