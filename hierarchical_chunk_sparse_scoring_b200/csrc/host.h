// Host-side helpers shared by the files that implement the C ABI.
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "hils.h"

namespace hils {

constexpr size_t kAlign = 256;
constexpr size_t kStatusBytes = 256;

inline size_t align_up(size_t x) { return (x + kAlign - 1) / kAlign * kAlign; }

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

inline bool ok_ptr(const void* ptr, bool needed) { return !needed || (ptr && aligned16(ptr)); }

inline hils_status check_device() {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return HILS_ERR_CUDA;
  int major = 0, minor = 0;
  if (cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev) != cudaSuccess)
    return HILS_ERR_CUDA;
  if (major != 10 || minor != 0) return HILS_ERR_UNSUPPORTED;
  return HILS_OK;
}

}  // namespace hils
