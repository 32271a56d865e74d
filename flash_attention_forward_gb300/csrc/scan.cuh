// Sums over the threads of a block.
#pragma once

#include <cuda_runtime.h>

namespace sdpa {

// Inclusive sum of v over the block's threads so far (before: the sum of earlier calls); total: the
// sum of all of them.  Two barriers.
__device__ __forceinline__ long long block_scan(long long v, long long before, long long (&warp_sum)[33], long long& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const long long y = __shfl_up_sync(0xffffffffu, v, d);
    if (lane >= d) v += y;
  }
  __syncthreads();
  if (lane == 31) warp_sum[warp] = v;
  __syncthreads();
  long long s = warp_sum[lane];  // every warp scans the 32 sums itself
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const long long y = __shfl_up_sync(0xffffffffu, s, d);
    if (lane >= d) s += y;
  }
  total = before + __shfl_sync(0xffffffffu, s, 31);
  const long long prev = __shfl_sync(0xffffffffu, s, warp > 0 ? warp - 1 : 0);
  return before + v + (warp > 0 ? prev : 0);
}

}  // namespace sdpa
