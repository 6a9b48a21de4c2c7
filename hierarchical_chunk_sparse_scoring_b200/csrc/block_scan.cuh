// Exclusive sum over a block of NT threads, one 64-bit value per thread.
#pragma once

#include <stdint.h>

namespace hils {

// sWarp: NT / 32 words of shared memory; `total` is the block's sum.  Called by every thread.
template <int NT>
__device__ __forceinline__ int64_t block_scan(int64_t v, int64_t* sWarp, int64_t& total) {
  constexpr int NW = NT / 32;
  static_assert(NT % 32 == 0 && NW <= 32, "whole warps, their sums in one warp");
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int64_t x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) sWarp[warp] = x;
  __syncthreads();
  // every warp sums the warps itself
  int64_t w = lane < NW ? sWarp[lane] : 0;
#pragma unroll
  for (int o = 1; o < NW; o <<= 1) {
    const int64_t y = __shfl_up_sync(0xffffffffu, w, o);
    if (lane >= o) w += y;
  }
  total = __shfl_sync(0xffffffffu, w, NW - 1);
  const int64_t before = __shfl_sync(0xffffffffu, w, warp ? warp - 1 : 0);
  __syncthreads();
  return (warp ? before : 0) + x - v;
}

}  // namespace hils
