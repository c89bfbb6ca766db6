// abi_util.h -- what the two halves of the C ABI (abi.hip, i8_abi.hip) share:
// the check of the current device, pointer alignment, and the outcome of a launch.
#pragma once

#include <hip/hip_runtime.h>

#include <atomic>
#include <cstring>

#include "gemmq.h"

namespace gemmq {

constexpr int kMaxDevices = 64;

// GEMMQ_OK when the current device is a gfx950 (looked up once per device).
inline int check_device() {
  static std::atomic<int> arch_ok[kMaxDevices];  // 0 unknown, 1 gfx950, 2 other
  int dev = -1;
  if (hipGetDevice(&dev) != hipSuccess || dev < 0) return GEMMQ_E_DEVICE;
  if (dev >= kMaxDevices) return GEMMQ_E_DEVICE;
  int state = arch_ok[dev].load(std::memory_order_acquire);
  if (state == 0) {
    hipDeviceProp_t prop;
    if (hipGetDeviceProperties(&prop, dev) != hipSuccess) return GEMMQ_E_DEVICE;
    state = std::strncmp(prop.gcnArchName, "gfx950", 6) == 0 ? 1 : 2;
    arch_ok[dev].store(state, std::memory_order_release);
  }
  return state == 1 ? GEMMQ_OK : GEMMQ_E_DEVICE;
}

inline bool aligned(const void* p, uintptr_t a) {
  return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0;
}

// Launcher outcome: -1 means the shape does not fit the kernel's launch
// geometry, -2 that the runtime refused a per-device kernel attribute; the
// callers check both before enqueuing anything, so here they only guard the
// launchers' own checks.  The thread's pending HIP error is cleared just before
// each launch (see clear_pending), so an error read here belongs to our launch.
inline int launched(int rc) {
  if (rc == -1) return GEMMQ_E_SHAPE;
  if (rc != 0) return GEMMQ_E_LAUNCH;
  return hipGetLastError() == hipSuccess ? GEMMQ_OK : GEMMQ_E_LAUNCH;
}

inline void clear_pending() { (void)hipGetLastError(); }

}  // namespace gemmq
