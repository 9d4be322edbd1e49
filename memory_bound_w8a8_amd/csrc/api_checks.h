// Host-side argument checks shared by the C entry points.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <atomic>
#include <cstring>

#include "fp8bq.h"

namespace fp8bq {

constexpr int64_t kMaxElems = int64_t(1) << 40;  // bound on M*K, N*K, M*N
constexpr int kMaxDevices = 64;

// Per-device capability cache: 0 = unknown, 1 = gfx950, -1 = not usable.
inline std::atomic<int> g_device_ok[kMaxDevices];

inline int check_device() {
  int dev = -1;
  if (hipGetDevice(&dev) != hipSuccess || dev < 0) return FP8BQ_ERR_DEVICE;
  if (dev >= kMaxDevices) return FP8BQ_ERR_DEVICE;
  int state = g_device_ok[dev].load(std::memory_order_acquire);
  if (state == 0) {
    hipDeviceProp_t prop;
    state = -1;
    if (hipGetDeviceProperties(&prop, dev) == hipSuccess && std::strncmp(prop.gcnArchName, "gfx950", 6) == 0)
      state = 1;
    g_device_ok[dev].store(state, std::memory_order_release);
  }
  return state == 1 ? FP8BQ_OK : FP8BQ_ERR_DEVICE;
}

inline bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

inline bool product_ok(int64_t a, int64_t b) { return a == 0 || b <= kMaxElems / a; }

inline int launch_status(hipError_t e) { return e == hipSuccess ? FP8BQ_OK : FP8BQ_ERR_LAUNCH; }

}  // namespace fp8bq
