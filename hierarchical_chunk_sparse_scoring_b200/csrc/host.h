// Host-side helpers shared by the files that implement the C ABI.
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include <atomic>

#include "hils.h"

namespace hils {

constexpr size_t kAlign = 256;
constexpr size_t kStatusBytes = 256;

inline size_t align_up(size_t x) { return (x + kAlign - 1) / kAlign * kAlign; }

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

inline bool ok_ptr(const void* ptr, bool needed) { return !needed || (ptr && aligned16(ptr)); }

// SMs of the current device if it is an sm_100 device, else 0; -1 if CUDA does not answer.  Looked
// up once per device (constants of the hardware).
inline int device_sms() {
  constexpr int kDevices = 64;
  static std::atomic<int> known[kDevices];   // SMs + 1
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return -1;
  if (dev >= 0 && dev < kDevices) {
    const int n = known[dev].load(std::memory_order_relaxed);
    if (n > 0) return n - 1;
  }
  int major = 0, minor = 0, sms = 0;
  if (cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return -1;
  if (major != 10 || minor != 0) sms = 0;
  if (dev >= 0 && dev < kDevices) known[dev].store(sms + 1, std::memory_order_relaxed);
  return sms;
}

inline hils_status check_device() {
  const int sms = device_sms();
  return sms < 0 ? HILS_ERR_CUDA : sms == 0 ? HILS_ERR_UNSUPPORTED : HILS_OK;
}

}  // namespace hils
