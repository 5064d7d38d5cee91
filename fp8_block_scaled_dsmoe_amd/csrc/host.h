// Host-side helpers of the C ABI sources.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include <atomic>
#include <cstring>

#include "dsmoe.h"

namespace dsmoe {

constexpr int64_t kI32Max = 2147483647LL;

inline bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

inline size_t round_up(size_t v, size_t a) { return (v + a - 1) / a * a; }

inline dsmoe_status launch_status(hipError_t e) { return e == hipSuccess ? DSMOE_OK : DSMOE_ERR_LAUNCH; }

inline bool valid_dtype(int t) { return t == DSMOE_BF16 || t == DSMOE_F32; }

// Device check, cached per device ordinal (idempotent).
inline std::atomic<int> g_dev_ok[64];

inline dsmoe_status check_device() {
  int dev = -1;
  if (hipGetDevice(&dev) != hipSuccess || dev < 0) return DSMOE_ERR_DEVICE;
  if (dev < 64) {
    const int v = g_dev_ok[dev].load(std::memory_order_relaxed);
    if (v == 1) return DSMOE_OK;
    if (v == 2) return DSMOE_ERR_DEVICE;
  }
  hipDeviceProp_t prop;
  if (hipGetDeviceProperties(&prop, dev) != hipSuccess) return DSMOE_ERR_DEVICE;
  const bool ok = std::strncmp(prop.gcnArchName, "gfx950", 6) == 0;
  if (dev < 64) g_dev_ok[dev].store(ok ? 1 : 2, std::memory_order_relaxed);
  return ok ? DSMOE_OK : DSMOE_ERR_DEVICE;
}

}  // namespace dsmoe
