// page_plan.cuh -- block tables and slot maps of a paged cache, built on the GPU from lengths.
//
// A step adds new[b] tokens to request b, which holds len[b] (new[b] < 0: the request has ended
// and gives its pages back).  With page size S, have = ceil(len / S), want = ceil((len + new) / S)
// and need = want - have pages; requests take pages in their order from the front of a ring of
// free pages, and released pages go behind the free ones.  Request b is admitted iff its table row
// is wide enough and need[b] = 0 or the running sum of need up to and with b is at most the number
// of free pages; the running sum never falls, so the admitted takers are a prefix of the takers
// and a request's first page is found from the exclusive sum alone.  A ring without room for all
// released pages keeps the first cap - count of them; the rest are lost, none is free twice.
//
// One launch: every CTA computes the three prefix sums over all requests itself (B integers from
// L2; a second launch or a device-wide barrier would cost more than the reads) and keeps them in
// shared memory; then all CTAs share the tokens (a binary search over the token offsets each),
// the table entries and the released pages.  No CTA reads what another one writes: new table
// entries are taken from the ring, not read back, ring entries that are read lie in
// [head, head + count) and those written behind it, and lengths and state go to new buffers.
// A step of 8 requests takes 2.9 us, of 1000 requests and 46,000 tokens 4.8: latencies, of the scan (two
// passes over the lengths) and of the search and dependent loads of each token.  With 45 of the requests
// ended it is 9.3: a warp copies such a request's pages, up to 1024 here, 32 at a time, and each round's
// loads wait for the stores of the one before.
#pragma once

#include <cstdint>

#include "rope.cuh"

namespace exattn {

constexpr int kPlanThreads = 512;
constexpr int kPlanMaxBatch = 16384;  // three prefix arrays of B + 1 ints in shared memory

struct PlanArgs {
  const int* lens;       // [B]
  const int* new_lens;   // [B]
  int* table;            // [B, width]
  int* queue;            // [cap] ring of free pages
  const int* state;      // {head, count}
  int* lens_out;         // [B]
  int* offsets;          // [B + 1]
  int* positions;        // [T]
  int* slots;            // [T]
  int* state_out;        // {head, count}
  int b, width, cap, page_shift, t;
};

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

__global__ void __launch_bounds__(kPlanThreads) page_plan_kernel(const PlanArgs a) {
  extern __shared__ int plan_smem[];
  int* s_tok = plan_smem;              // [b + 1] first token of each request
  int* s_need = plan_smem + a.b + 1;   // [b] first free page taken, or -1: not admitted
  int* s_back = s_need + a.b;          // [b] first place of a released request's pages
  __shared__ int warp_sums[kPlanThreads / 32][3];
  __shared__ int s_taken;
  if (threadIdx.x == 0) s_taken = 0;
  grid_launch_dependents();
  grid_wait();

  int head = a.state[0], count = a.state[1];
  count = min(max(count, 0), a.cap);
  head = static_cast<int>(static_cast<unsigned>(head) % static_cast<unsigned>(a.cap));
  const int limit = a.width << a.page_shift;  // at most 2^30
  // a request's length as far as its table row can hold it
  auto length = [&](int r) { return min(max(a.lens[r], 0), limit); };
  auto pages = [&](int tokens) { return tokens ? ((tokens - 1) >> a.page_shift) + 1 : 0; };
  auto wants = [&](int r, int len, int add) {
    return static_cast<long long>(len) + add <= limit ? pages(len + add) - pages(len) : -1;
  };

  const int per = (a.b + kPlanThreads - 1) / kPlanThreads;
  const int r0 = min(a.b, static_cast<int>(threadIdx.x) * per), r1 = min(a.b, r0 + per);
  int v[3] = {0, 0, 0}, total[3];
  for (int r = r0; r < r1; ++r) {
    const int len = length(r), add = a.new_lens[r];
    v[0] += max(add, 0);
    v[1] += max(wants(r, len, max(add, 0)), 0);
    v[2] += add < 0 ? pages(len) : 0;
  }
  block_scan3(v, total, warp_sums);
  int taken = 0;
  for (int r = r0; r < r1; ++r) {
    const int len = length(r), add = a.new_lens[r];
    const int want = wants(r, len, max(add, 0)), need = max(want, 0);
    const bool ok = want == 0 || (want > 0 && v[1] + need <= count);
    s_tok[r] = v[0];
    s_need[r] = ok ? v[1] : -1;
    s_back[r] = v[2];
    if (ok && need > 0) taken = v[1] + need;
    v[0] += max(add, 0);
    v[1] += need;
    v[2] += add < 0 ? pages(len) : 0;
  }
  if (threadIdx.x == 0) s_tok[a.b] = total[0];
  if (taken > 0) atomicMax(&s_taken, taken);  // an integer maximum: any order gives the same
  __syncthreads();

  const int gthread = blockIdx.x * kPlanThreads + threadIdx.x;
  const int gthreads = gridDim.x * kPlanThreads;
  // place i <= cap of the ring, counted from its head
  auto ring = [&](int i) {
    const unsigned x = static_cast<unsigned>(head) + static_cast<unsigned>(i), cap = static_cast<unsigned>(a.cap);
    return static_cast<int>(x >= cap ? x - cap : x);
  };
  if (gthread == 0) {
    a.state_out[0] = ring(s_taken);
    // released pages count as far as they were stored: the places past `cap`, counted from the head, hold
    // the pages that this step hands out
    a.state_out[1] = count - s_taken + min(total[2], a.cap - count);
  }
  for (int r = gthread; r <= a.b; r += gthreads) {
    a.offsets[r] = s_tok[r];
    if (r == a.b) continue;
    const int len = length(r), add = a.new_lens[r];
    a.lens_out[r] = add < 0 ? 0 : (s_need[r] >= 0 ? len + add : len);
  }
  // table entries of admitted requests and pages of ended ones, a warp per request
  const int lane = threadIdx.x % 32;
  for (int r = gthread / 32; r < a.b; r += gthreads / 32) {
    const int len = length(r), add = a.new_lens[r];
    const int have = pages(len);
    int* row = a.table + static_cast<long long>(r) * a.width;
    if (add < 0) {
      for (int i = lane; i < have; i += 32) {
        const long long at = static_cast<long long>(count) + s_back[r] + i;
        if (at < a.cap) a.queue[ring(static_cast<int>(at))] = row[i];
      }
    } else if (s_need[r] >= 0) {
      const int need = pages(len + add) - have;
      for (int i = lane; i < need; i += 32)
        row[have + i] = a.queue[ring(s_need[r] + i)];
    }
  }
  for (int t = gthread; t < a.t; t += gthreads) {
    int pos = 0, slot = -1;
    // (tokens that number 2^31 or more wrap: then a place may be found that is not the token's)
    if (t < total[0]) {
      int lo = 0, hi = a.b;  // the last request whose first token is at or before t
      while (hi - lo > 1) {
        const int mid = (lo + hi) / 2;
        if (s_tok[mid] <= t) lo = mid; else hi = mid;
      }
      const int len = length(lo);
      pos = len + (t - s_tok[lo]);
      if (s_need[lo] >= 0 &&
          static_cast<unsigned>(t - s_tok[lo]) < static_cast<unsigned>(s_tok[lo + 1] - s_tok[lo])) {
        const int p = pos >> a.page_shift, have = pages(len);
        const int id = p < have ? a.table[static_cast<long long>(lo) * a.width + p]
                                : a.queue[ring(s_need[lo] + p - have)];
        // an id that no cache has: its slot would wrap into another page
        if (id >= 0 && id <= 0x7fffffff >> a.page_shift)
          slot = (id << a.page_shift) + (pos & ((1 << a.page_shift) - 1));
      }
    }
    a.positions[t] = pos;
    a.slots[t] = slot;
  }
}

}  // namespace exattn
