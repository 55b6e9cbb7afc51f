// block_scan.cuh -- prefix sums over the requests of a step, which page planning and acceptance share.
#pragma once

#include <cstdint>

namespace exattn {

constexpr int kPlanThreads = 512;
constexpr int kPlanMaxBatch = 16384;  // three prefix arrays of B + 1 ints in shared memory

// Exclusive prefix sums over the block's threads of three values, and their totals.
__device__ __forceinline__ void block_scan3(int (&v)[3], int (&total)[3], int (*warp_sums)[3]) {
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  int inc[3];
#pragma unroll
  for (int k = 0; k < 3; ++k) {
    inc[k] = v[k];
#pragma unroll
    for (int o = 1; o < 32; o *= 2) {
      const int x = __shfl_up_sync(0xffffffffu, inc[k], o);
      if (lane >= o) inc[k] += x;
    }
    if (lane == 31) warp_sums[warp][k] = inc[k];
  }
  __syncthreads();
#pragma unroll
  for (int k = 0; k < 3; ++k) {
    int before = 0, all = 0;
    for (int w = 0; w < kPlanThreads / 32; ++w) {
      const int x = warp_sums[w][k];
      before += w < warp ? x : 0;
      all += x;
    }
    total[k] = all;
    v[k] = before + inc[k] - v[k];
  }
  __syncthreads();
}

}  // namespace exattn
