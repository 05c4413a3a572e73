// What the host sides of the library share: the HIP error text behind
// carve_error_string and the dynamic-LDS limits raised so far.
#pragma once
#include <hip/hip_runtime.h>

#include <atomic>
#include <cstdint>

#include "carve.h"

namespace carve_host {

// Records `e` for carve_error_string(CARVE_EHIP) on this thread and returns CARVE_EHIP.
__attribute__((visibility("hidden"))) int hip_failed(hipError_t e);

inline size_t elem_bytes(int dtype) { return dtype == CARVE_F32 ? 4 : 2; }
inline bool misaligned(const void* p) { return p && (reinterpret_cast<uintptr_t>(p) & 15u); }
inline bool misaligned4(const void* p) { return reinterpret_cast<uintptr_t>(p) & 3u; }   // int32 and single fp32
inline bool overlaps(const void* a, size_t na, const void* b, size_t nb) {
  if (!a || !b || na == 0 || nb == 0) return false;
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return x < y + nb && y < x + na;
}

// Raises kernel Kern's dynamic-LDS limit to `bytes`. The attribute only ever
// needs raising, so the largest value set so far is kept per kernel (one
// instantiation of this function per kernel) and device, and the driver is
// called only to go beyond it: later calls (and launches inside a graph
// capture) make no attribute call at all.
constexpr int kMaxDevices = 64;
template <auto Kern>
hipError_t set_lds(int bytes) {
  static std::atomic<int> set_bytes[kMaxDevices];
  auto raise = [&] {
    return hipFuncSetAttribute(reinterpret_cast<const void*>(Kern),
                               hipFuncAttributeMaxDynamicSharedMemorySize, bytes);
  };
  int dev = -1;
  if (hipGetDevice(&dev) != hipSuccess || dev < 0 || dev >= kMaxDevices) return raise();
  int cur = set_bytes[dev].load(std::memory_order_acquire);
  if (cur >= bytes) return hipSuccess;
  const hipError_t e = raise();
  if (e != hipSuccess) return e;
  while (cur < bytes && !set_bytes[dev].compare_exchange_weak(cur, bytes, std::memory_order_acq_rel)) {
  }
  return hipSuccess;
}

}  // namespace carve_host
