// Host helpers of the entry points' files: refusals, alignment and overlap of arguments, the device, launch errors.
#pragma once
#include <atomic>
#include <cstdint>
#include <cstdio>

#include "common.cuh"
#include "gdn.h"

namespace gdn {

inline int bad(const char* msg) { return set_last_error(GDN_EINVAL, msg); }
inline size_t align256(size_t x) { return (x + 255) & ~size_t(255); }
inline bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

// Whether [a, a + na) and [b, b + nb) share a byte.
inline bool overlap(const void* a, size_t na, const void* b, size_t nb) {
  const char *x = static_cast<const char*>(a), *y = static_cast<const char*>(b);
  return a && b && x < y + nb && y < x + na;
}

// The current device is a GB300: asked of the driver once per device and process.
inline int device_or_error(int* sms) {
  static std::atomic<int> known[64];  // SM count of a supported device, 0 before the first question
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return set_last_error(GDN_EUNSUPPORTED, "no CUDA device");
  if (dev < 64) n = known[dev].load(std::memory_order_relaxed);
  if (!n) {
    if (gdn_device_supported(dev) != GDN_OK)
      return set_last_error(GDN_EUNSUPPORTED, "device is not compute capability 10.3 (GB300)");
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
      return set_last_error(GDN_ECUDA, "SM count query failed");
    if (dev < 64) known[dev].store(n, std::memory_order_relaxed);
  }
  if (sms) *sms = n;
  return GDN_OK;
}

inline int cuda_rc(cudaError_t e, const char* what) {
  if (e == cudaSuccess) return GDN_OK;
  char msg[256];
  snprintf(msg, sizeof(msg), "%s: %s", what, cudaGetErrorString(e));
  return set_last_error(GDN_ECUDA, msg);
}

}  // namespace gdn
