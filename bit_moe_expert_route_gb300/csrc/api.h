// What the C entry points' argument checks share (host side).
#pragma once

#include <atomic>
#include <cstdint>
#include <cuda_runtime.h>

#include "moe.h"

namespace moe {

inline bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

inline int cuda_status(cudaError_t e) {
  if (e == cudaSuccess) return MOE_OK;
  (void)cudaGetLastError();  // clear a non-sticky launch error
  return MOE_ERR_CUDA;
}

// The current device's SM count, or a status < 0. The attributes are looked
// up once a device (they are most of a small call's time on the host).
inline int device_sms() {
  constexpr int kMaxDev = 64;
  static std::atomic<int> known[kMaxDev];  // 0 = not looked up
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return MOE_ERR_CUDA;
  if (dev >= 0 && dev < kMaxDev) {
    const int v = known[dev].load(std::memory_order_relaxed);
    if (v) return v;
  }
  int major = 0, minor = 0, sms = 0;
  if (cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return MOE_ERR_CUDA;
  const int r = major == 10 && minor == 3 ? sms : MOE_ERR_ARCH;
  if (dev >= 0 && dev < kMaxDev) known[dev].store(r, std::memory_order_relaxed);
  return r;
}

}  // namespace moe
