// Host-side checks shared by the C entry points: alignment, overlap, size
// arithmetic, the device check and the launch status.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>
#include <string.h>

#include <atomic>

#include "nvfp4.h"

namespace nvfp4_abi {

constexpr int64_t kMaxDevices = 64;
inline std::atomic<int> g_device_ok[kMaxDevices];  // 0 unknown, 1 gfx950, 2 other

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// [a, a+na) and [b, b+nb) overlap (byte ranges).
inline bool overlaps(const void* a, int64_t na, const void* b, int64_t nb) {
  const uintptr_t pa = reinterpret_cast<uintptr_t>(a), pb = reinterpret_cast<uintptr_t>(b);
  return na > 0 && nb > 0 && pa < pb + (uintptr_t)nb && pb < pa + (uintptr_t)na;
}

// a * b fits in int64 (a, b >= 0).
inline bool mul_ok(int64_t a, int64_t b, int64_t* out) {
  if (a != 0 && b > INT64_MAX / a) return false;
  *out = a * b;
  return true;
}

// Checks that the current device is a gfx950 (cached per device).
inline nvfp4_status check_device() {
  int dev = 0;
  if (hipGetDevice(&dev) != hipSuccess) return NVFP4_ERR_DEVICE;
  if (dev < 0 || dev >= kMaxDevices) return NVFP4_ERR_DEVICE;
  int st = g_device_ok[dev].load(std::memory_order_relaxed);
  if (st == 0) {
    hipDeviceProp_t prop;
    if (hipGetDeviceProperties(&prop, dev) != hipSuccess) return NVFP4_ERR_DEVICE;
    st = (strncmp(prop.gcnArchName, "gfx950", 6) == 0) ? 1 : 2;
    g_device_ok[dev].store(st, std::memory_order_relaxed);
  }
  return st == 1 ? NVFP4_OK : NVFP4_ERR_UNSUPPORTED;
}

inline nvfp4_status launch_status() { return hipGetLastError() == hipSuccess ? NVFP4_OK : NVFP4_ERR_DEVICE; }

}  // namespace nvfp4_abi
