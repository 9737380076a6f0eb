// Prefix sums over the requests of a batch, by one block.
#pragma once
#include <cstdint>

namespace dsa {

// Exclusive prefix sum of v over the block's THREADS threads; *total gets the
// sum.  warp_sums: THREADS / 32 entries of shared memory.
template <int THREADS>
__device__ __forceinline__ int64_t block_scan(int64_t v, int64_t* total, int64_t* warp_sums) {
  constexpr int kWarps = THREADS / 32;
  static_assert(THREADS % 32 == 0 && kWarps <= 32, "one warp sums the warps");
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int64_t s = v;
#pragma unroll
  for (int o = 1; o < 32; o *= 2) {
    const int64_t t = __shfl_up_sync(0xffffffffu, s, o);
    if (lane >= o) s += t;
  }
  __syncthreads();               // an earlier scan's sums have been read
  if (lane == 31) warp_sums[warp] = s;
  __syncthreads();
  if (warp == 0) {
    int64_t x = lane < kWarps ? warp_sums[lane] : 0;
#pragma unroll
    for (int o = 1; o < 32; o *= 2) {
      const int64_t t = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += t;
    }
    if (lane < kWarps) warp_sums[lane] = x;
  }
  __syncthreads();
  *total = warp_sums[kWarps - 1];
  return (warp == 0 ? 0 : warp_sums[warp - 1]) + s - v;
}

// The last index i in [0, n) with start[i] <= x (start rises from 0): the
// request whose range holds x (empty ranges share a start with the next one).
__device__ __forceinline__ int scan_owner(const int32_t* start, int n, int x) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (start[mid] <= x) lo = mid;
    else hi = mid;
  }
  return lo;
}

}  // namespace dsa
