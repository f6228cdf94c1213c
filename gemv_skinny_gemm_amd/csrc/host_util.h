// host_util.h - host-side checks shared by the cache's and the verification's
// source files: the current device, pointer alignment and buffer overlap.  The
// linears' source has its own: bench.py reports HBM traffic from the counters on
// record only while that file is the one that they were taken on.
#ifndef SKINNY_HOST_UTIL_H
#define SKINNY_HOST_UTIL_H

#include <hip/hip_runtime.h>

#include <stddef.h>
#include <stdint.h>
#include <string.h>

#include <mutex>

#include "skinny_gemm.h"

namespace skinny_host {

struct DeviceInfo {
  int cus = 0;
  bool gfx950 = false;
  bool valid = false;
};

constexpr int kMaxDevices = 64;
inline DeviceInfo g_dev[kMaxDevices];
inline std::mutex g_dev_mu;

// Properties of the current device, cached on first use.
inline skinny_status device_info(DeviceInfo* out) {
  int dev = 0;
  if (hipGetDevice(&dev) != hipSuccess) return SKINNY_ERR_HIP;
  if (dev < 0 || dev >= kMaxDevices) return SKINNY_ERR_UNSUPPORTED;
  std::lock_guard<std::mutex> lock(g_dev_mu);
  if (!g_dev[dev].valid) {
    hipDeviceProp_t p;
    if (hipGetDeviceProperties(&p, dev) != hipSuccess) return SKINNY_ERR_HIP;
    g_dev[dev].cus = p.multiProcessorCount;
    g_dev[dev].gfx950 = strncmp(p.gcnArchName, "gfx950", 6) == 0;
    g_dev[dev].valid = true;
  }
  *out = g_dev[dev];
  return SKINNY_OK;
}

inline bool aligned(const void* p, size_t a) { return ((uintptr_t)p % a) == 0; }

struct Range {
  uintptr_t lo, hi;
};

inline bool overlap(Range a, Range b) { return a.lo < b.hi && b.lo < a.hi; }

inline Range range_of(const void* p, size_t bytes) {
  return Range{(uintptr_t)p, (uintptr_t)p + bytes};
}

}  // namespace skinny_host

#endif  // SKINNY_HOST_UTIL_H
