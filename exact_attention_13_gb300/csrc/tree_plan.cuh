// tree_plan.cuh -- bookkeeping of trees of drafted tokens: positions and masks before the step that checks
// them, and what of them is accepted after it.
//
// A request brings n nodes behind its len cached tokens; node i hangs on node parent(i) < i of the same
// request, or (parent -1) on the last cached token.  With A(i) = {i} and A(parent(i)), the nodes on the way
// up from i,
//     position(i) = len + |A(i)| - 1,      node i sees the cached tokens and the nodes of A(i).
// A(i) is kept as bits, 32 nodes a word.
//
// Plan.  A block takes a request; its nodes' bits and pointers lie in shared memory and double their reach
// each round: A(i) |= A(up(i)), up(i) = up(up(i)), so a chain of n nodes takes log2(n) rounds instead of n
// dependent loads.  Rounds end when every pointer has left the tree.  8 requests of 9 nodes take 2.6 us, 1000 of
// 64 4.3: the latencies of a launch, two dependent loads and the rounds' barriers.
//
// Acceptance.  choice(i) is the token that the model chose behind node i.  Node 0 of a request holds the token
// that was chosen before, and is good; another one is good if its token is its parent's choice (of several
// such children the first).  A node is accepted iff all of A(i) is good, that is, iff A(i) without the good
// nodes is empty: no walk down the tree.  The accepted nodes are a path, and node i's place on it is
// |A(i)| - 1.  The pages behind the new lengths are given back in the requests' order, which needs the sums over all
// requests: up to kTreeGroups requests a CTA and eight CTAs do all of it in one cluster; larger batches take a
// second kernel, launched while the first runs.
//
// 1000 requests of 64 nodes take 6.0 us, the second kernel under the end of the first.
//
// Integers only: results do not depend on scheduling (the one atomic is a minimum).
#pragma once

#include <cstdint>

#include "block_scan.cuh"
#include "rope.cuh"

namespace exattn {

constexpr int kTreeThreads = 128;
constexpr int kTreeNodes = 256;  // nodes of a request that others can see, 32 a word
constexpr int kTreeWords = kTreeNodes / 32;

// A request's first node and the nodes there are of it (offsets are device data: kept inside the buffers).
struct TreeShape {
  int first, n;
};
__device__ __forceinline__ TreeShape tree_shape(const int* offsets, int r, int t) {
  const int first = min(max(offsets[r], 0), t);
  return {first, min(max(offsets[r + 1], first), t) - first};
}

struct TreePlanArgs {
  const int* parents;    // [T]
  const int* offsets;    // [B + 1]
  const int* lens;       // [B]
  int* positions;        // [T]
  uint32_t* seen;        // [T, words]
  int b, t, words;
};

__global__ void __launch_bounds__(kTreeThreads) tree_plan_kernel(const TreePlanArgs a) {
  __shared__ uint32_t s_seen[kTreeNodes][kTreeWords + 1];
  __shared__ int s_up[kTreeNodes];
  grid_launch_dependents();
  grid_wait();
  const int tid = threadIdx.x, r = blockIdx.x;
  if (r >= a.b) {  // rows behind the last request
    const int from = min(max(a.offsets[a.b], 0), a.t), step = (gridDim.x - a.b) * kTreeThreads;
    for (int t = from + (r - a.b) * kTreeThreads + tid; t < a.t; t += step) {
      a.positions[t] = 0;
      for (int w = 0; w < a.words; ++w) a.seen[static_cast<size_t>(t) * a.words + w] = 0u;
    }
    return;
  }
  const TreeShape s = tree_shape(a.offsets, r, a.t);
  const int n = min(s.n, 32 * a.words);  // nodes that have bits
  const int len = a.lens[r];
  auto parent = [&](int i) {
    const int p = a.parents[s.first + i];
    return p < i ? p : -1;
  };
  constexpr int kPer = kTreeNodes / kTreeThreads;
#pragma unroll
  for (int x = 0; x < kPer; ++x) {
    const int i = x * kTreeThreads + tid;
    if (i < n) {
      s_up[i] = parent(i);
      for (int w = 0; w < a.words; ++w) s_seen[i][w] = w == i / 32 ? 1u << (i % 32) : 0u;
    }
  }
  // (at most log2(n) rounds: pointers fall by doubling distances)
  while (true) {
    int up[kPer], next[kPer];
    uint32_t more[kPer][kTreeWords];
    bool any = false;
    __syncthreads();
#pragma unroll
    for (int x = 0; x < kPer; ++x) {
      const int i = x * kTreeThreads + tid;
      up[x] = i < n ? s_up[i] : -1;
      if (up[x] >= 0) {
        any = true;
        next[x] = s_up[up[x]];
#pragma unroll
        for (int w = 0; w < kTreeWords; ++w)
          if (w < a.words) more[x][w] = s_seen[up[x]][w];
      }
    }
    if (!__syncthreads_or(any)) break;
#pragma unroll
    for (int x = 0; x < kPer; ++x) {
      const int i = x * kTreeThreads + tid;
      if (up[x] >= 0) {
        s_up[i] = next[x];
#pragma unroll
        for (int w = 0; w < kTreeWords; ++w)
          if (w < a.words) s_seen[i][w] |= more[x][w];
      }
    }
  }
  auto write = [&](int i, int depth, auto bits) {
    uint32_t* const out = a.seen + static_cast<size_t>(s.first + i) * a.words;
    for (int w = 0; w < a.words; ++w) {
      out[w] = bits(w);
      if (i < n) depth += __popc(out[w]);
    }
    a.positions[s.first + i] = static_cast<int>(static_cast<unsigned>(len) + static_cast<unsigned>(depth));
  };
  for (int i = tid; i < n; i += kTreeThreads) write(i, -1, [&](int w) { return s_seen[i][w]; });
  // Nodes past the bits are seen by none: they take the bits of the nodes above them that have some.  128 at a time, their
  // pointers double until they leave the 128 for a node that has its results, or for none.
  int* const s_hops = reinterpret_cast<int*>(s_seen);  // [128] steps that the pointer stands for
  for (int i0 = n; i0 < s.n; i0 += kTreeThreads) {
    const int i = i0 + tid;
    __syncthreads();
    if (i < s.n) {
      s_up[tid] = parent(i);
      s_hops[tid] = 1;
    }
    for (int reach = 1; reach < kTreeThreads; reach *= 2) {
      __syncthreads();
      const int up = i < s.n ? s_up[tid] : -1;
      int next = 0, hops = 0;
      if (up >= i0) {
        next = s_up[up - i0];
        hops = s_hops[up - i0];
      }
      __syncthreads();
      if (up >= i0) {
        s_up[tid] = next;
        s_hops[tid] += hops;
      }
    }
    if (i < s.n) {
      const int up = s_up[tid];
      const uint32_t* const above = a.seen + static_cast<size_t>(s.first + max(up, 0)) * a.words;
      const int depth = up < 0 ? -1 : a.positions[s.first + up] - len;
      write(i, depth + s_hops[tid], [&](int w) { return up < 0 ? 0u : above[w]; });
    }
  }
}

struct TreeAcceptArgs {
  const int* parents;    // [T]
  const uint32_t* seen;  // [T, words]
  const int* tokens;     // [T]
  const int* choices;    // [T]
  const int* lens;       // [B] before the step
  const int* after;      // [B] with the nodes
  const int* offsets;    // [B + 1]
  const int* slots;      // [T]
  const int* table;      // [B, width]
  int* queue;            // [cap]
  const int* state;      // {head, count}
  int* lens_out;         // [B]
  int* counts;           // [B]
  int* path;             // [T]
  int* next;             // [B]
  int* sources;          // [T]
  int* state_out;        // {head, count}
  int b, t, words, width, cap, page_shift;
};

// Barriers of 128 threads of the CTA.
__device__ __forceinline__ void group_sync(int group) {
  asm volatile("barrier.cta.sync.aligned %0, %1;" ::"r"(group + 1), "n"(kTreeThreads) : "memory");
}
__device__ __forceinline__ int group_count(int group, bool yes) {
  int n;
  asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %3, 0;\n\tbarrier.cta.red.popc.aligned.u32 %0, %1, %2, p;\n\t}"
               : "=r"(n)
               : "r"(group + 1), "n"(kTreeThreads), "r"(static_cast<unsigned>(yes))
               : "memory");
  return n;
}

struct TreeAcceptGroup {
  int choice[kTreeNodes], slot[kTreeNodes], first[kTreeNodes], path[kTreeNodes];
  uint32_t good[kTreeWords];
};

// Request r, by a group of 128 threads of the CTA.
__device__ __forceinline__ void accept_request(const TreeAcceptArgs& a, TreeAcceptGroup& g, int r, int group) {
  int(&s_choice)[kTreeNodes] = g.choice, (&s_slot)[kTreeNodes] = g.slot, (&s_first)[kTreeNodes] = g.first,
  (&s_path)[kTreeNodes] = g.path;
  uint32_t(&s_good)[kTreeWords] = g.good;
  const int tid = threadIdx.x % kTreeThreads, lane = tid % 32;
  const TreeShape s = tree_shape(a.offsets, r, a.t);
  const int before = a.lens[r], after = a.after[r];
  const int n = after > before ? min(s.n, 32 * a.words) : 0;  // a refused request has no places
  constexpr int kPer = kTreeNodes / kTreeThreads;
  int parent[kPer], token[kPer];
  uint32_t seen[kPer][kTreeWords];
#pragma unroll
  for (int x = 0; x < kPer; ++x) {
    const int i = x * kTreeThreads + tid;
    if (i < n) {
      parent[x] = a.parents[s.first + i];
      token[x] = a.tokens[s.first + i];
      s_choice[i] = a.choices[s.first + i];
      s_slot[i] = a.slots[s.first + i];
      s_first[i] = kTreeNodes;
      s_path[i] = 0;
#pragma unroll
      for (int w = 0; w < kTreeWords; ++w)
        seen[x][w] = w < a.words ? a.seen[static_cast<size_t>(s.first + i) * a.words + w] : 0u;
    }
  }
  group_sync(group);
  bool hit[kPer];
#pragma unroll
  for (int x = 0; x < kPer; ++x) {
    const int i = x * kTreeThreads + tid;
    hit[x] = i < n && parent[x] >= 0 && parent[x] < i && token[x] == s_choice[parent[x]];
    if (hit[x]) atomicMin(&s_first[parent[x]], i);
  }
  group_sync(group);
#pragma unroll
  for (int x = 0; x < kPer; ++x) {
    const int i = x * kTreeThreads + tid;
    const bool good = (i == 0 && n > 0) || (hit[x] && s_first[parent[x]] == i);
    const unsigned word = __ballot_sync(0xffffffffu, good);
    if (lane == 0) s_good[i / 32] = word;
  }
  group_sync(group);
  int count = 0;
#pragma unroll
  for (int x = 0; x < kPer; ++x) {
    const int i = x * kTreeThreads + tid;
    bool on = i < n;
    int place = -1;
    if (on) {
#pragma unroll
      for (int w = 0; w < kTreeWords; ++w) {
        on = on && (seen[x][w] & ~s_good[w]) == 0u;
        place += __popc(seen[x][w]);
      }
      if (on && place >= 0) s_path[place] = i;
    }
    count += group_count(group, on);
  }
  for (int i = tid; i < s.n; i += kTreeThreads) {
    const int node = i < count ? min(max(s_path[i], 0), n - 1) : -1;
    a.path[s.first + i] = node;
    a.sources[s.first + i] = node >= 0 ? s_slot[node] : -1;
  }
  if (tid == 0) {
    a.counts[r] = count;
    a.next[r] = count > 0 ? s_choice[min(max(s_path[count - 1], 0), n - 1)] : -1;
    a.lens_out[r] = min(before, after) + count;
  }
}

// Rows behind the last request.
__device__ __forceinline__ void accept_no_request(const TreeAcceptArgs& a, int thread, int threads) {
  for (int t = min(max(a.offsets[a.b], 0), a.t) + thread; t < a.t; t += threads) a.path[t] = a.sources[t] = -1;
}

// Pages of a length, up to those of the table, and the ones that the request gives back.
__device__ __forceinline__ int tree_pages(const TreeAcceptArgs& a, int tokens) {
  return tokens > 0 ? ((min(tokens, a.width << a.page_shift) - 1) >> a.page_shift) + 1 : 0;  // (at most 2^30 tokens)
}
__device__ __forceinline__ int tree_back(const TreeAcceptArgs& a, int r) {
  return max(tree_pages(a, a.after[r]) - tree_pages(a, __ldcg(a.lens_out + r)), 0);
}
// The ring's free pages before: from `head` on, `count` of them.
struct TreeRing {
  int head, count;
};
__device__ __forceinline__ TreeRing tree_ring(const TreeAcceptArgs& a) {
  return {static_cast<int>(static_cast<unsigned>(a.state[0]) % static_cast<unsigned>(a.cap)), min(max(a.state[1], 0), a.cap)};
}
__device__ __forceinline__ void tree_ring_out(const TreeAcceptArgs& a, const TreeRing& ring, int total) {
  a.state_out[0] = ring.head;
  a.state_out[1] = ring.count + min(total, a.cap - ring.count);
}
// Request r's n pages, behind `before` ones of other requests (a warp).
__device__ __forceinline__ void give_back(const TreeAcceptArgs& a, const TreeRing& ring, int r, int n, int before) {
  const int* const row = a.table + static_cast<long long>(r) * a.width + tree_pages(a, __ldcg(a.lens_out + r));
  for (int i = threadIdx.x % 32; i < n; i += 32) {
    const long long at = static_cast<long long>(ring.count) + before + i;
    if (at >= a.cap) continue;  // a ring without room for all keeps the first ones
    const unsigned x = static_cast<unsigned>(ring.head) + static_cast<unsigned>(at), cap = static_cast<unsigned>(a.cap);
    a.queue[x >= cap ? x - cap : x] = row[i];
  }
}

// Up to kTreeGroups requests a CTA, all of the batch's in a cluster: acceptance and pages (8 requests: 3.4 us
// against 4.0 by two kernels, 64: 4.2 and 4.1, and a call from Python 26 against 29).
constexpr int kTreeGroups = 8, kTreeCluster = 8;
__global__ void __launch_bounds__(kTreeGroups* kTreeThreads) tree_accept_small_kernel(const TreeAcceptArgs a) {
  __shared__ TreeAcceptGroup groups[kTreeGroups];
  grid_launch_dependents();
  grid_wait();
  const int group = threadIdx.x / kTreeThreads, r = blockIdx.x * kTreeGroups + group;
  if (r < a.b) accept_request(a, groups[group], r, group);
  const int threads = gridDim.x * kTreeGroups * kTreeThreads;
  accept_no_request(a, blockIdx.x * kTreeGroups * kTreeThreads + threadIdx.x, threads);
  // every CTA's lengths are there for all
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
  const TreeRing ring = tree_ring(a);
  const int lane = threadIdx.x % 32, warp = blockIdx.x * (kTreeGroups * kTreeThreads / 32) + threadIdx.x / 32;
  if (warp >= a.b) return;
  // warp i has request i; pages of the ones before it, two requests a lane
  static_assert(kTreeGroups * kTreeCluster <= 64, "requests of a cluster");
  int mine = 0, before = 0, total = 0;
#pragma unroll
  for (int x = 0; x < 64; x += 32) {
    const int q = x + lane, n = q < a.b ? tree_back(a, q) : 0;
    total += n;
    before += q < warp ? n : 0;
    mine += q == warp ? n : 0;
  }
  total = __reduce_add_sync(0xffffffffu, total);
  before = __reduce_add_sync(0xffffffffu, before);
  mine = __reduce_add_sync(0xffffffffu, mine);
  if (warp == 0 && lane == 0) tree_ring_out(a, ring, total);
  give_back(a, ring, warp, mine, before);
}

// Any batch: a request a CTA, one more for the rows behind the last request.
__global__ void __launch_bounds__(kTreeThreads) tree_accept_kernel(const TreeAcceptArgs a) {
  __shared__ TreeAcceptGroup one;
  grid_launch_dependents();
  grid_wait();
  if (static_cast<int>(blockIdx.x) < a.b)
    accept_request(a, one, blockIdx.x, 0);
  else
    accept_no_request(a, threadIdx.x, kTreeThreads);
}

// The pages behind the new lengths go behind the free ones of the ring, in the requests' order (as in
// page_plan_kernel: every CTA sums over all requests itself).
__global__ void __launch_bounds__(kPlanThreads) tree_release_kernel(const TreeAcceptArgs a) {
  extern __shared__ int plan_smem[];
  int* const s_back = plan_smem;  // [b] first place of a request's released pages
  __shared__ int warp_sums[kPlanThreads / 32][3];
  grid_launch_dependents();
  grid_wait();
  const TreeRing ring = tree_ring(a);
  const int per = (a.b + kPlanThreads - 1) / kPlanThreads;
  const int r0 = min(a.b, static_cast<int>(threadIdx.x) * per), r1 = min(a.b, r0 + per);
  int v[3] = {0, 0, 0}, total[3];
  for (int r = r0; r < r1; ++r) v[0] += tree_back(a, r);
  block_scan3(v, total, warp_sums);
  for (int r = r0; r < r1; ++r) {
    s_back[r] = v[0];
    v[0] += tree_back(a, r);
  }
  __syncthreads();
  const int gthread = blockIdx.x * kPlanThreads + threadIdx.x, gthreads = gridDim.x * kPlanThreads;
  if (gthread == 0) tree_ring_out(a, ring, total[0]);
  for (int r = gthread / 32; r < a.b; r += gthreads / 32) give_back(a, ring, r, tree_back(a, r), s_back[r]);
}

}  // namespace exattn
