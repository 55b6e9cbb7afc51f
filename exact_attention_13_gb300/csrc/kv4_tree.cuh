// kv4_tree.cuh -- attention of trees of drafted tokens over the paged 4-bit cache.
//
// The operation of kv4_attn.cuh with another mask: a node sees the keys before its request's tree, and of the
// tree's keys those whose bit is set in its row of `seen`.  Units of N = 32 or 64 query rows (one key head of
// one request, rows ordered by node, then by head of the group).
//
// Both products take the widened cache as the 128-row operand of tcgen05.mma, out of tensor memory:
//     S^T [128 keys x N] = K [128 x d] Q^T,      O^T [d x N] += V^T [d x 128 keys] P^T
// so the tensor core does N products a cached value (query rows as the 128-row operand: 128, mostly padding),
// and the widened tiles, four times the cache's bytes, go from registers to tensor memory without
// a write and a read of shared memory.  What is left there a tile is the codes (written once by asynchronous copies, read
// once), Q^T (N x d, read by the product) and P^T (128 x N).
//
// Layouts.  An A operand in tensor memory is one lane a row and 32 bits of two neighbouring contraction indices a
// column.  Contraction indices and rows may be permuted freely, so the tiles are stored with the 16x128b shape:
// thread (g, t) = (lane / 4, lane % 4) writes rows g and g + 8, columns 4 n + t.
//   K: column 4 n + t holds dims t d/4 + 2 n and the next one: a thread reads d/4 neighbouring codes of a row.
//      Row m holds key 16 (t' + 4 (n' % 2)) + 2 (n' / 2) + e with m = 8 n' + 2 t' + e.
//   V^T: column 4 n + t holds keys 16 (t + 4 (n % 2)) + 2 (n / 2) and the next one, that is, contraction index k holds
//      the key of row m = k of K: a thread of the softmax writes P of its own key to row m of P^T.  Row 32 q + 8 i + g
//      is dim 32 q + 4 g + i (d = 128; for d = 64 row 32 q + 8 i + g, i < 2, is dim 16 q + 2 g + i and the other rows
//      are not used): a thread needs 4 neighbouring codes, 16 bits, of each of its keys.  For d = 128 a warp loads eight
//      keys' 16 bytes at a time, one key of each group of 16 (whose codes are padded to other banks), and movmatrix
//      transposes the 8 x 8 matrix of 16-bit pieces.
//
// Softmax.  A thread has one key and N/2 rows, so a row's sum runs over threads: each keeps partial sums of its
// keys, added up at the end of a unit.  The maximum would be one reduction a tile, row and warp; instead the
// reference m of a row is moved only when some score of the tile lies more than 2^15 above it (kDecLazy): a
// maximum over the thread's own scores and one barrier with a vote decide, and mostly nothing else happens.
//
// Roles (640 threads, one CTA a SM):
//   warps 0-7    softmax: lanes 32 (w % 4) .. + 31 (keys; dims of O^T), rows N/2 (w / 4) .. + N/2 - 1; outputs
//   warps 8-15   widen K and V^T: two warps share 32 rows of both
//   warp  16     issues the MMAs:  S(0) S(1) | PV(t) S(t + 2) | ...
//   warps 17, 18 copy codes and scales of K and of V into a ring of tiles
//   warp  19     queries, masks and places of the rows of the next unit, while this one runs (the first unit's are
//                brought by the softmax warps)
// The split over CTAs and the merge of units that cross them are those of kv4_attn.cuh.
//
// Copies go by 16 bytes a lane: a bulk copy takes its issuer about 90 cycles whatever its size, and a tile has 32
// pieces.  The two issue orders that would overlap more (PV and S from warps of their own; three steps in
// flight with 24 warps) were not faster.
//
// Measured (64 requests of 4096 keys, 8 key heads, d 128: 302 MB of cache, 44 us at 6.8 TB/s): 123 us for 32 rows of a
// key head, 141 us for 64; 1800 to 2000 cycles a tile of 128 keys, of which the copies are 800.  Bound by neither
// memory (0.36 and 0.31 of its rate) nor the tensor core (0.15 and 0.25) but by the hand-offs copy - widen - S -
// softmax - PV of the tiles and, three to four times a CTA, of the units: with copies, widening, exponentials and
// MMAs all left out the waits and the units' work alone took 71 and 97 us.  What was worth the most on the way (64
// rows, 269 us at first): masks by node in shared memory instead of by row (a word a row and tile before), one
// exponent for all rows' queries, code small enough for the instruction cache (its placement alone moves the 32
// rows between 123 and 131 us).
//
// Every mbarrier wait is bounded in time; one that runs out sets the CTA's abort flag and the status word, and
// all roles leave.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cstdint>

#include "fa_fwd_kernel.cuh"
#include "kv4_attn.cuh"
#include "kv4_chunk.cuh"
#include "tree_plan.cuh"

namespace exattn {

constexpr int kTrThreads = 640;
constexpr int kTrKeys = 128;
constexpr int kTrMmaWarp = 16, kTrCopyWarp = 17, kTrQueryWarp = 19;
// 640 threads get 96 registers each at launch; softmax 256 x 120 + widening 256 x 80 + the others 128 x 80
constexpr int kTrLaunchRegs = 96, kTrSoftmaxRegs = 120, kTrWidenRegs = 80, kTrOtherRegs = 80;
static_assert(256 * kTrSoftmaxRegs + 256 * kTrWidenRegs + 128 * kTrOtherRegs == kTrThreads * kTrLaunchRegs,
              "registers of the block at launch");
constexpr int kTrFlags = 32;  // tiles whose flags are kept: more than are ever between copies and softmax

template <int D, int N>
struct TreeGeo {
  // a stage of the ring: codes of K, of V (16 keys at a time, padded by 16 bytes), scales of K, of V
  static constexpr int kGroup = 16 * D / 2, kVGroup = kGroup + 16, kScales = 16 * D / 16;
  static constexpr int kV = 8 * kGroup, kKs = kV + 8 * kVGroup, kVs = kKs + 8 * kScales, kStage = kVs + 8 * kScales;
  static constexpr int kStages = 8;
  static constexpr int kQBytes = N * D * 2;             // boxes of 64 dims, 128 bytes a row
  static constexpr int kPBytes = 128 * 128;             // a row of 128 bytes a key
  static constexpr int kO = 2 * N, kK = 3 * N, kVt = kK + 2 * (D / 2);  // columns behind the two S
  static_assert(kVt + 2 * 64 <= 512, "tensor memory");
  static constexpr uint32_t kIdescS = instr_desc(128, N, 0, false, false);
  static constexpr uint32_t kIdescPV = instr_desc(128, N, 0, false, true);
  static constexpr int kHalf = N / 2;                   // rows of a softmax thread
  static_assert(N == 32 || N == 64, "rows of a unit");
};

// A share of a unit: tiles [tile, tile + n) of its `tiles`; n = 0: there are no more.
struct TreeSeg {
  int r, head, block, tile, n, tiles;
  ReqShape req;
};
struct TreeWalk {
  TreeSeg s;
  int blocks;
  long long left;  // of the CTA's share behind the segment
};

template <int N>
struct TreeRows {          // of one unit, written by the query warps
  TreeSeg seg;
  float c;                 // factor of the scores
  int apart;               // rows have factors of their own, which every tile's scores get first
  float row_c[N];
  float most[N], down[N];  // of the queries: the rows' largest values (the first unit's), what they are multiplied by
  int out[N];              // row of o and lse, -1: padding
  uint32_t seen[kTreeNodes][N / 32];  // rows that see a node
};

template <int N>
struct TreeCtrl {
  uint64_t ring_full[8], ring_empty[8];
  uint64_t k_full[2], v_full[2], s_full[2], p_full[2], pv_done[2];
  uint64_t q_full[2], q_empty[2], o_empty, drain;
  uint32_t tmem_base;
  int abort;
  int flags[kTrFlags];     // bit g: 16-key group g of the tile is there; -1: no more tiles
  long long sum[32];
  long long total, first, last;
  int extra, skip;         // what a unit counts more on the line, and how much of that the share begins with
  TreeSeg start;
  TreeRows<N> rows[2];
  alignas(16) float nm[N];  // minus the reference of a row's probabilities
  float alpha[N];
  float top[4][N];          // of each quarter's keys: maxima, and in the end sums
  alignas(16) uint32_t scales[8][8][12];  // V's scales of a widening warp, as pairs of keys
};

template <int D, int N>
constexpr int tree_smem_bytes() {
  using G = TreeGeo<D, N>;
  return 2 * G::kQBytes + 2 * G::kPBytes + G::kStages * G::kStage + static_cast<int>(sizeof(TreeCtrl<N>)) + 1024;
}

// ---- small PTX
// Whether three phases have all completed; does not wait.
__device__ __forceinline__ uint32_t mbar_test3(uint32_t b0, uint32_t p0, uint32_t b1, uint32_t p1, uint32_t b2,
                                               uint32_t p2) {
  uint32_t done;
  asm volatile(
      "{\n\t.reg .pred q0, q1, q2;\n\t"
      "mbarrier.test_wait.parity.shared::cta.b64 q0, [%1], %2;\n\t"
      "mbarrier.test_wait.parity.shared::cta.b64 q1, [%3], %4;\n\t"
      "mbarrier.test_wait.parity.shared::cta.b64 q2, [%5], %6;\n\t"
      "and.pred q0, q0, q1;\n\tand.pred q0, q0, q2;\n\t"
      "selp.u32 %0, 1, 0, q0;\n\t}"
      : "=r"(done)
      : "r"(b0), "r"(p0), "r"(b1), "r"(p1), "r"(b2), "r"(p2)
      : "memory");
  return done;
}
// The largest of the warp's values (NaN: the others).
__device__ __forceinline__ float warp_max(float v) {
  float y;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(y) : "f"(v));
  return y;
}
// An arrival on `bar` when the thread's copies so far have landed.
__device__ __forceinline__ void cp_async_arrive(uint32_t bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
}
// Barrier over `threads` threads that tells whether any of them votes yes.
__device__ __forceinline__ bool bar_any(int id, int threads, bool vote) {
  uint32_t any;
  __syncwarp();
  asm volatile("{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %3, 0;\n\t"
               "barrier.cta.red.or.pred.aligned q, %1, %2, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
               : "=r"(any)
               : "r"(id), "r"(threads), "r"(static_cast<uint32_t>(vote))
               : "memory");
  return any != 0;
}
__device__ __forceinline__ void bar_wait(int id, int threads) {
  asm volatile("barrier.cta.sync.aligned %0, %1;" ::"r"(id), "r"(threads) : "memory");
}
#define EXATTN_R4(r, i) "=r"(r[i]), "=r"(r[i + 1]), "=r"(r[i + 2]), "=r"(r[i + 3])
#define EXATTN_W4(r, i) "r"(r[i]), "r"(r[i + 1]), "r"(r[i + 2]), "r"(r[i + 3])
// N consecutive columns of the thread's lane.
template <int N>
__device__ __forceinline__ void tmem_ld_cols(uint32_t taddr, uint32_t (&r)[N]) {
  static_assert(N == 8 || N == 16 || N == 32, "columns of one load");
  if constexpr (N == 8)  // (maxima of eight rows at a time)
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : EXATTN_R4(r, 0), EXATTN_R4(r, 4)
                 : "r"(taddr));
  if constexpr (N == 16)
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, "
                 "%14, %15}, [%16];"
                 : EXATTN_R4(r, 0), EXATTN_R4(r, 4), EXATTN_R4(r, 8), EXATTN_R4(r, 12)
                 : "r"(taddr));
  if constexpr (N == 32) tmem_ld32(taddr, r);
}
template <int N>
__device__ __forceinline__ void tmem_st_cols(uint32_t taddr, const uint32_t (&r)[N]) {
  static_assert(N == 8 || N == 16 || N == 32, "columns of one store");
  if constexpr (N == 8)  // (scores of rows apart)
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(taddr),
                 EXATTN_W4(r, 0), EXATTN_W4(r, 4)
                 : "memory");
  if constexpr (N == 16) tmem_st16(taddr, r);
  if constexpr (N == 32) tmem_st32(taddr, r);
}
// 16 lanes from the address's on, 32 columns: r[2 n + i] to row lane / 4 + 8 i, column 4 n + lane % 4.
__device__ __forceinline__ void tmem_st_16x128b_x8(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile("tcgen05.st.sync.aligned.16x128b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, "
               "%14, %15, %16};" ::"r"(taddr),
               EXATTN_W4(r, 0), EXATTN_W4(r, 4), EXATTN_W4(r, 8), EXATTN_W4(r, 12)
               : "memory");
}
// 16 lanes from the address's on: r[2 n + i] from row lane / 4 + 8 i, column 4 n + lane % 4.
template <int N>
__device__ __forceinline__ void tmem_ld_16x128b(uint32_t taddr, uint32_t (&r)[N]) {
  static_assert(N == 8 || N == 16, "registers of one load");
  if constexpr (N == 8)
    asm volatile("tcgen05.ld.sync.aligned.16x128b.x4.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : EXATTN_R4(r, 0), EXATTN_R4(r, 4)
                 : "r"(taddr));
  if constexpr (N == 16)
    asm volatile("tcgen05.ld.sync.aligned.16x128b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, "
                 "%14, %15}, [%16];"
                 : EXATTN_R4(r, 0), EXATTN_R4(r, 4), EXATTN_R4(r, 8), EXATTN_R4(r, 12)
                 : "r"(taddr));
}
#undef EXATTN_R4
#undef EXATTN_W4

// ---- the line of tiles
template <int N>
__device__ __forceinline__ int tree_blocks(const Kv4Args& a, const ReqShape& s) {
  return static_cast<int>((static_cast<long long>(s.q_len) * a.group + N - 1) / N);
}
__device__ __forceinline__ int tree_tiles(const ReqShape& s) { return max(1, (s.keys - 1) / kTrKeys + 1); }

// On the line of tiles that the CTAs share a unit counts `extra` more than it has, at its front: queries, first
// reference, sums and outputs take the time of that many tiles (64 requests of 500 to 8192 keys, up to 64 rows: 187 us with
// 0, 160 with 4 or 6, 166 with 8; of 16 to 2048 keys 75 with 4, 67 with 6, 68 with 8; 32 rows: 47.5, 49.4, 51.3).  A share
// that ends among them leaves the whole unit to the next one.  Where the CTAs have few tiles each, spreading them is
// worth more.  Units that are not split count 1.
template <int N>
__device__ __forceinline__ int tree_extra(const Kv4Args& a, long long tiles) {
  return !a.whole_tiles && tiles >= 16ll * gridDim.x ? (N == 64 ? 6 : 4) : 0;
}
// Tiles of the walk's unit that its share has, from s.tile on, after `skip` of the line in front of them.
__device__ __forceinline__ void tree_take(const Kv4Args& a, TreeWalk& w, int skip) {
  if (a.whole_tiles) {
    w.s.n = w.left > 0 ? w.s.tiles : 0;
    w.left -= 1;
  } else {
    w.left -= skip;
    w.s.n = static_cast<int>(max(0ll, min(static_cast<long long>(w.s.tiles - w.s.tile), w.left)));
    w.left -= w.s.n;
  }
}
// The next segment of a warp's walk (every lane does the same); s.n = 0 at the end of the share.
template <int N>
__device__ __forceinline__ void tree_next(const Kv4Args& a, const TreeCtrl<N>* ctl, TreeWalk& w) {
  w.s.n = 0;
  if (w.left <= 0) return;
  w.s.tile = 0;
  if (++w.s.head == a.hk) {
    w.s.head = 0;
    if (++w.s.block == w.blocks) {
      w.s.block = 0;
      do {
        ++w.s.r;
        w.s.req = kv4_request(a, w.s.r);
        w.blocks = tree_blocks<N>(a, w.s.req);
      } while (w.blocks == 0 && w.s.r + 1 < a.b);
      w.s.tiles = tree_tiles(w.s.req);
    }
  }
  tree_take(a, w, ctl->extra);
}
template <int N>
__device__ __forceinline__ TreeWalk tree_walk(const Kv4Args& a, const TreeCtrl<N>* ctl) {
  TreeWalk w;
  w.s = ctl->start;
  w.blocks = tree_blocks<N>(a, w.s.req);
  w.left = ctl->last - ctl->first;
  tree_take(a, w, ctl->skip);
  return w;
}

// The CTA's share [first, last) of the line of `total`; fills ctl->start.  Returns the number of CTAs that have work.
template <int N>
__device__ __forceinline__ int tree_my_range(const Kv4Args& a, TreeCtrl<N>* ctl) {
  const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32;
  ReqShape s{0, 0, 0, 0};
  int per = 1, extra = 0;
  long long units = 0;  // of the thread's requests
  auto cost = [&](int r) -> long long {
    if (r >= a.b) return 0;
    s = kv4_request(a, r);
    per = a.whole_tiles ? 1 : tree_tiles(s) + extra;
    const long long u = static_cast<long long>(tree_blocks<N>(a, s)) * a.hk;
    units += u;
    return u * per;
  };
  // inclusive scan over the block; ctl->sum keeps the warps' sums until the next barrier
  auto scan = [&](long long x) {
#pragma unroll
    for (int o = 1; o < 32; o *= 2) {
      const long long y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    if (lane == 31) ctl->sum[warp] = x;
    __syncthreads();
#pragma unroll 1
    for (int w = 0; w < warp; ++w) x += ctl->sum[w];
    return x;
  };
  auto all_sum = [&]() {
    long long x = 0;
#pragma unroll 1
    for (int w = 0; w < kTrThreads / 32; ++w) x += ctl->sum[w];
    return x;
  };
  long long mine = 0, tiles = 0;
  for (int r = tid; r < a.b; r += kTrThreads) mine += tiles = cost(r);
  long long inc = scan(mine), total = all_sum();
  extra = tree_extra<N>(a, total);
  if (extra > 0) {  // the line again, with what each unit counts more
    per += extra;
    tiles += extra * units;  // (up to one request a thread: the scan below is the line itself)
    __syncthreads();
    inc = scan(mine + extra * units);
    total = all_sum();
  }
  const int n = static_cast<int>(min(static_cast<long long>(gridDim.x), total));
  if (static_cast<int>(blockIdx.x) >= n) {
    __syncthreads();
    return n;
  }
  const long long first = share_begin(total, n, blockIdx.x), last = share_begin(total, n, blockIdx.x + 1);
  long long base = 0;
  for (int r0 = 0; r0 < a.b; r0 += kTrThreads) {
    long long all = total;
    if (a.b > kTrThreads) {
      __syncthreads();
      tiles = cost(r0 + tid);
      inc = scan(tiles) + base;
      all = base + all_sum();
    }
    if (first >= inc - tiles && first < inc) {
      const long long off = first - (inc - tiles);
      // (64-bit divisions take about 100 instructions)
      const int u = off <= 0x7fffffffll ? static_cast<int>(off) / per : static_cast<int>(off / per);
      const int block = u / a.hk;
      const int at = a.whole_tiles ? 0 : static_cast<int>(off - static_cast<long long>(u) * per);
      ctl->start = TreeSeg{r0 + tid, u - block * a.hk, block, max(0, at - extra), 0, tree_tiles(s), s};
      ctl->skip = max(0, extra - at);
      ctl->extra = extra;
      ctl->total = total;
      ctl->first = first;
      ctl->last = last;
    }
    base = all;
    if (first < base) break;
  }
  __syncthreads();
  return n;
}

template <int D, int N>
__global__ void __launch_bounds__(kTrThreads, 1) kv4_tree_kernel(const Kv4Args a) {
  using G = TreeGeo<D, N>;
  extern __shared__ __align__(1024) uint8_t tr_smem[];
  uint8_t* const smem =
      reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(tr_smem) + 1023) & ~static_cast<uintptr_t>(1023));
  uint8_t* const s_q = smem;
  uint8_t* const s_p = smem + 2 * G::kQBytes;
  uint8_t* const s_ring = s_p + 2 * G::kPBytes;
  static_assert(G::kStages * G::kStage % 16 == 0 && G::kQBytes % 1024 == 0, "alignment");
  TreeCtrl<N>* const ctl = reinterpret_cast<TreeCtrl<N>*>(s_ring + G::kStages * G::kStage);
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;

  grid_launch_dependents();
  if (warp == kTrMmaWarp) {
    tmem_alloc(smem_u32(&ctl->tmem_base), 512);
    tmem_relinquish();
  }
  if (threadIdx.x == 0) {
    for (int i = 0; i < G::kStages; ++i) {
      mbar_init(smem_u32(&ctl->ring_full[i]), 65);  // the copying warps' lanes, and the flags
      mbar_init(smem_u32(&ctl->ring_empty[i]), 8);  // one arrival per widening warp
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_u32(&ctl->k_full[i]), 8);
      mbar_init(smem_u32(&ctl->v_full[i]), 8);
      mbar_init(smem_u32(&ctl->s_full[i]), 1);
      mbar_init(smem_u32(&ctl->p_full[i]), 8);   // one arrival per softmax warp
      mbar_init(smem_u32(&ctl->pv_done[i]), 1);
      mbar_init(smem_u32(&ctl->q_full[i]), 1);
      mbar_init(smem_u32(&ctl->q_empty[i]), 9);  // the unit's last S, and the softmax warps
    }
    mbar_init(smem_u32(&ctl->o_empty), 8);
    mbar_init(smem_u32(&ctl->drain), 1);
    ctl->abort = 0;
    fence_mbar_init();
  }
  tc_fence_before();
  const int n_cta = tree_my_range<N>(a, ctl);  // (ends with a barrier)
  tc_fence_after();
  const uint32_t tmem = ctl->tmem_base;
  if (static_cast<int>(blockIdx.x) >= n_cta) {
    if (threadIdx.x == 0 && !a.whole_tiles) a.desc[blockIdx.x] = make_int4(-1, 0, 0, 0);
    if (warp == kTrMmaWarp) tmem_dealloc(tmem, 512);
    return;
  }
  volatile int* const abort_flag = &ctl->abort;
  // For the number-th completion, counted from 0.  The first try that fails starts the clock, and a wait that runs out
  // raises the CTA's abort flag (small code: there are 20 copies of it).
  auto wait = [&](uint64_t& bar, int number) -> bool {
    const uint32_t at = smem_u32(&bar), parity = static_cast<uint32_t>(number) & 1u;
    uint64_t limit = 0;
#pragma unroll 1
    while (!__all_sync(0xffffffffu, mbar_try_wait(at, parity))) {
      const uint64_t now = globaltimer_ns();
      if (limit == 0) limit = now + kWaitLimitNs;
      if (__any_sync(0xffffffffu, *abort_flag || now > limit)) {
        *abort_flag = 1;
        return false;
      }
    }
    return true;
  };

  // ---- a unit's queries: they come by 16 bytes to where the row's operand lies and are turned into it in place
  constexpr int kPieces = D / 8, kRowsIt = 32 / kPieces, kLanes = D / 32;
  auto piece_at = [&](int buffer, int row, int piece) {
    return buffer * G::kQBytes + piece / 8 * (N * 128) + row * 128 + ((piece % 8 ^ (row & 7)) << 4);
  };
  auto fetch = [&](int buffer, int row0, long long at) {  // kRowsIt rows; at: the lane's row in q, -1: zeros
    const int piece = lane % kPieces;
    cp_async16(smem_u32(s_q) + piece_at(buffer, row0 + lane / kPieces, piece), a.q + (at < 0 ? 0 : at + piece * 8),
               at < 0 ? 0u : 16u);
  };
  auto row_most = [&](int buffer, int row, int first, int step) {  // largest finite value of a row's pieces first, ...
    __nv_bfloat162 top = __float2bfloat162_rn(0.f);
#pragma unroll 4
    for (int x = first; x < kPieces; x += step) {
      const uint4 raw = *reinterpret_cast<const uint4*>(s_q + piece_at(buffer, row, x));
      const __nv_bfloat162* const v = reinterpret_cast<const __nv_bfloat162*>(&raw);
#pragma unroll
      for (int e = 0; e < 4; ++e)  // (infinities and NaN: 0 x + |x| is NaN, and the maximum the other one)
        top = __hmax2(top, __hfma2(v[e], __float2bfloat162_rn(0.f), __habs2(v[e])));
    }
    return fmaxf(__low2float(top), __high2float(top));
  };
  // A power of two brings the largest finite value of all rows into [2^14, 2^15), so that the softmax needs one factor
  // for all of them.  Rows whose largest lies 2^13 below have a power of their own (f16 then holds bf16's 8 bits down to
  // 2^-18 of any row's largest at least), and all rows' scores get their factors ahead of the softmax.  So they do
  // where they may pass 2^26: what the reference of such a row is rounded by would leave f16's range in a
  // fused multiplication and difference.
  auto factors = [&](TreeRows<N>& rows, const float (&most)[N / 32]) {  // of rows lane, lane + 32
    float amax = most[0];
#pragma unroll
    for (int x = 1; x < N / 32; ++x) amax = fmaxf(amax, most[x]);
    amax = warp_max(amax);
    const uint32_t all_ex = __float_as_uint(amax) >> 23, all_down = min(268u - all_ex, 253u);
    constexpr float kMost = 448.f * 6.f * D;  // of a product with a vector of ones
    bool apart = amax * a.c * kMost > 0x1p26f;
#pragma unroll
    for (int x = 0; x < N / 32; ++x) {
      const uint32_t ex = __float_as_uint(most[x]) >> 23;
      const bool own = most[x] > 0.f && ex + 13u < all_ex;
      const uint32_t down = own ? min(268u - ex, 253u) : all_down;
      apart |= own;
      rows.down[x * 32 + lane] = __uint_as_float(down << 23);
      rows.row_c[x * 32 + lane] = a.c * __uint_as_float((254u - down) << 23);
    }
    apart = __any_sync(0xffffffffu, apart);
    if (lane == 0) {
      rows.apart = apart;
      rows.c = apart ? 1.f : a.c * __uint_as_float((254u - all_down) << 23);
    }
  };
  // 32 / kLanes rows: a lane takes d/4 dims of a row, 8 of each quarter, which are four chunks of the operand
  auto convert = [&](int buffer, const TreeRows<N>& rows, int row, bool mine) {
    const int part = lane % kLanes;
    uint32_t h[4][4];
    if (mine) {
      const float down = rows.down[row];
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        float f[8];
        unpack_bf16x8(*reinterpret_cast<const uint4*>(s_q + piece_at(buffer, row, x * kLanes + part)), f);
#pragma unroll
        for (int e = 0; e < 4; ++e) h[x][e] = pack_f16x2(f[2 * e] * down, f[2 * e + 1] * down);
      }
    }
    __syncwarp();
    if (mine) {
#pragma unroll
      for (int e = 0; e < 4; ++e)
        st_shared_v4(smem_u32(s_q) + piece_at(buffer, row, 4 * part + e), h[0][e], h[1][e], h[2][e], h[3][e]);
    }
  };
  struct RowPlace {
    long long from;  // in q, -1: padding
    int token, out;
  };
  auto place = [&](const TreeSeg& seg, int row) {
    const int at = seg.block * N + row, node = at / a.group;
    const int head = seg.head * a.group + at - node * a.group, token = seg.req.q0 + node;
    const bool live = at < seg.req.q_len * a.group;
    return RowPlace{live ? static_cast<long long>(token) * a.q_row + static_cast<long long>(head) * a.q_head : -1, token,
                    live ? token * a.hq + head : -1};
  };

  if (warp >= kTrMmaWarp) {
    regs_dec<kTrOtherRegs>();
    if (warp == kTrMmaWarp) {
      // ============================================================ MMA issuer
      const uint64_t q_desc = smem_desc(smem_u32(s_q), 16, 1024, kSwizzle128B);
      const uint64_t p_desc = smem_desc(smem_u32(s_p), 128 * 128, 1024, kSwizzle128B);
      // S(t + 2) is issued behind PV(t): what it overwrites, S(t), has been read when P(t) is there, so the step waits for
      // P(t), V(t) and K(t + 2) at once (a wait takes 150 cycles even if nothing is left to wait for), and S(t + 1) runs
      // under the softmax of tile t.  Its completion, behind PV(t)'s, tells the softmax that P's buffer is free.
      int u_s = -1, left_s = 0;  // the unit that S works on, and its tiles to come
      int u_v = -1, left_v = 0;
      bool ok = true;
      auto issue_s = [&](int t) {
        tc_fence_after();
        --left_s;
        if (elect_one()) {
          const uint64_t qd = q_desc + (u_s & 1) * (G::kQBytes >> 4);
          const uint32_t k = tmem + G::kK + (t & 1) * (D / 2), s = tmem + (t & 1) * N;
          mma_chain_ts_off<4, 0, 2, 8, 16, 24, 32, 40, 48, 56>(s, G::kIdescS, 0u, k, qd);
          if constexpr (D == 128)
            mma_chain_ts_off<4, 0, 2, 8, 16, 24, 32, 40, 48, 56>(s, G::kIdescS, 1u, k + 32, qd + (N * 128 >> 4));
          tc_commit(smem_u32(&ctl->s_full[t & 1]));
          if (left_s == 0) tc_commit(smem_u32(&ctl->q_empty[u_s & 1]));
        }
        __syncwarp();
      };
      int pv = 0, s_next = 0;
#pragma unroll 1
      for (bool more = true; ok && (more || pv < s_next);) {
        // (the first two passes issue S only)
        const bool with_pv = s_next - pv == 2 || !more, in_unit = more && left_s > 0;
        bool k_there = false;
        if (with_pv) {
          bool begins = false;
          if (left_v == 0) {
            ++u_v;
            left_v = ctl->rows[u_v & 1].seg.n;
            begins = true;
            if (u_v > 0) ok = wait(ctl->o_empty, u_v - 1);
          }
          --left_v;
          uint64_t &bp = ctl->p_full[pv & 1], &bv = ctl->v_full[pv & 1];
          uint64_t& bk = in_unit ? ctl->k_full[s_next & 1] : bv;
          const int nk = in_unit ? s_next >> 1 : pv >> 1;
          if (ok) {
            k_there = __all_sync(0xffffffffu, mbar_test3(smem_u32(&bp), pv >> 1 & 1, smem_u32(&bv), pv >> 1 & 1,
                                                         smem_u32(&bk), nk & 1));
            if (!k_there) ok = wait(bp, pv >> 1) && wait(bv, pv >> 1);
          }
          if (!ok) break;
          tc_fence_after();
          if (elect_one()) {
            mma_chain_ts_off<8, 0, 128, 8, 16, 24, 32, 40, 48, 56>(
                tmem + G::kO, G::kIdescPV, begins ? 0u : 1u, tmem + G::kVt + (pv & 1) * 64,
                p_desc + (pv & 1) * (G::kPBytes >> 4));
            tc_commit(smem_u32(&ctl->pv_done[pv & 1]));
          }
          __syncwarp();
          ++pv;
        }
        if (!more) continue;
        if (!in_unit) {
          ++u_s;
          ok = wait(ctl->q_full[u_s & 1], u_s >> 1);
          if (!ok) break;
          left_s = ctl->rows[u_s & 1].seg.n;
          more = left_s > 0;
          if (!more) continue;
        }
        if (!(k_there && in_unit)) ok = wait(ctl->k_full[s_next & 1], s_next >> 1);
        if (!ok) break;
        issue_s(s_next++);
      }
      // nothing this warp issued may still run when the TMEM is released
      __syncwarp();
      if (elect_one()) tc_commit(smem_u32(&ctl->drain));
      const uint64_t t0 = globaltimer_ns();
      while (!mbar_try_wait(smem_u32(&ctl->drain), 0) && globaltimer_ns() - t0 < kWaitLimitNs) {
      }
    } else if (warp < kTrQueryWarp) {
      // ============================================================ copies of the cache
      // 16 bytes a lane and copy.  Groups of 16 keys on pages that are not there are not copied: their scores are
      // masked, and whatever lies in the ring is a number after widening.
      TreeWalk w = tree_walk<N>(a, ctl);
      const int page_rows = 1 << a.page_shift;
      const int block_bytes = kv4_block_bytes(page_rows, D);
      const size_t page_bytes = static_cast<size_t>(block_bytes) * 2u * a.hk;
      const int self = warp - kTrCopyWarp;  // 0: keys, 1: values
      // scales: kJoin groups a copy, kLanes lanes each
      constexpr int kLanes = G::kScales / 16, kJoin = 32 / kLanes;
      const int sc_group = lane / kLanes, sc_at = lane % kLanes * 16;
      const uint32_t ring = smem_u32(s_ring);
      const uint32_t sc_dst = ring + (self ? G::kVs : G::kKs) + sc_group * G::kScales + sc_at;
      const uint32_t code_dst = ring + (self ? G::kV : 0) + lane * 16;
      const uint32_t group_step = self ? G::kVGroup : G::kGroup;
      const size_t sc_from = static_cast<size_t>(page_rows) * (D / 2) + sc_at;
      int t = 0;
      bool ok = true;
      while (w.s.n > 0 && ok && !EXATTN_INJECT_STALL) {
        const int* const ids = a.table + static_cast<size_t>(w.s.r) * a.width;
        const uint8_t* const head = a.cache + static_cast<size_t>(2 * w.s.head + self) * block_bytes;
        int key = w.s.tile * kTrKeys + lane % 8 * 16;  // lanes g, g + 8, ...: group g
        int id = key < w.s.req.keys ? ids[key >> a.page_shift] : -1;
        for (int i = 0; i < w.s.n; ++i, ++t) {
          const int next = key + kTrKeys;
          const int id_next = i + 1 < w.s.n && next < w.s.req.keys ? ids[next >> a.page_shift] : -1;
          const int slot = t % G::kStages;
          if (t >= G::kStages) ok = wait(ctl->ring_empty[slot], t / G::kStages - 1);
          if (!ok) break;
          const bool there = static_cast<unsigned>(id) < static_cast<unsigned>(a.pages);
          const int flags = static_cast<int>(__ballot_sync(0xffffffffu, there) & 0xffu);
          const size_t page_at = there ? static_cast<size_t>(id) * page_bytes : 0;
          const int row = key & (page_rows - 1);
          const uint32_t stage = slot * G::kStage;
#pragma unroll
          for (int g = 0; g < 8; ++g) {
            const uint8_t* const from = head + __shfl_sync(0xffffffffu, page_at + row * (D / 2), g) + lane * 16;
            if (flags >> g & 1) {
#pragma unroll
              for (int x = 0; x < G::kGroup; x += 512) cp_async16(code_dst + stage + g * group_step + x, from + x, 16u);
            }
          }
          const size_t scale_at = page_at + row * (D / 16);
#pragma unroll
          for (int g0 = 0; g0 < 8; g0 += kJoin) {
            const int g = g0 + sc_group;
            const uint8_t* const from = head + __shfl_sync(0xffffffffu, scale_at, g) + sc_from;
            if (flags >> g & 1) cp_async16(sc_dst + stage + g0 * G::kScales, from, 16u);
          }
          const uint32_t bar = smem_u32(&ctl->ring_full[slot]);
          cp_async_arrive(bar);
          if (self == 0 && lane == 0) {
            ctl->flags[t % kTrFlags] = flags;
            mbar_arrive(bar);
          }
          key = next;
          id = id_next;
        }
        if (ok) tree_next<N>(a, ctl, w);
      }
      if (ok) ok = t < G::kStages || wait(ctl->ring_empty[t % G::kStages], t / G::kStages - 1);
      if (ok && !EXATTN_INJECT_STALL) {  // (a test build delivers nothing: the first waits run out)
        const uint32_t bar = smem_u32(&ctl->ring_full[t % G::kStages]);
        if (self == 0 && lane == 0) {
          ctl->flags[t % kTrFlags] = -1;
          mbar_arrive(bar);
        }
        mbar_arrive(bar);
      }
      cp_async_commit();
      cp_async_wait<0>();  // copies under way land before the CTA's shared memory goes away
    } else {
      // ============================================================ queries, masks and places of a unit's rows
      TreeWalk w = tree_walk<N>(a, ctl);
      constexpr int kOffsets = N / 32;
      constexpr int kUnroll = N == 32 ? 2 : 1;  // (32 rows: 123 us with 2 and 131 with 1, 64 rows: 143 and 141)
      for (int u = 0;; ++u) {
        if (u == 0) {  // (the first unit's are brought by the softmax warps)
          tree_next<N>(a, ctl, w);
          continue;
        }
        if (u >= 2 && !wait(ctl->q_empty[u & 1], (u >> 1) - 1)) break;
        TreeRows<N>& rows = ctl->rows[u & 1];
        if (lane == 0) rows.seg = w.s;
        if (w.s.n > 0) {
          long long from[kOffsets];  // of rows lane, lane + 32
#pragma unroll
          for (int x = 0; x < kOffsets; ++x) {
            const RowPlace p = place(w.s, x * 32 + lane);
            from[x] = p.from;
            rows.out[x * 32 + lane] = p.out;
            // the lane's row of bits, a word at a time, becomes a bit of each node's word
#pragma unroll 1
            for (int y = 0; 32 * y < min(w.s.req.queries, 32 * a.words); ++y) {
              const uint32_t bits = p.out >= 0 ? a.tree[static_cast<size_t>(p.token) * a.words + y] : 0u;
              uint32_t mine = 0u;
#pragma unroll 4
              for (int e = 0; e < 32; ++e) {
                const uint32_t node = __ballot_sync(0xffffffffu, bits >> e & 1u);
                mine = lane == e ? node : mine;
              }
              rows.seen[32 * y + lane][x] = mine;
            }
          }
#pragma unroll 4
          for (int row0 = 0; row0 < N; row0 += kRowsIt) {
            const int row = row0 + lane / kPieces;
            fetch(u & 1, row0, __shfl_sync(0xffffffffu, kOffsets > 1 && row0 >= 32 ? from[kOffsets - 1] : from[0], row % 32));
          }
          cp_async_commit();
          cp_async_wait<0>();
          __syncwarp();
          float most[kOffsets];
#pragma unroll
          for (int x = 0; x < kOffsets; ++x) most[x] = row_most(u & 1, x * 32 + lane, 0, 1);
          factors(rows, most);
          __syncwarp();
#pragma unroll(kUnroll)
          for (int row0 = 0; row0 < N; row0 += 32 / kLanes) convert(u & 1, rows, row0 + lane / kLanes, true);
          fence_proxy_async_smem();  // the MMAs read the queries through the async proxy
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&ctl->q_full[u & 1]));
        if (w.s.n == 0) break;
        tree_next<N>(a, ctl, w);
      }
    }
  } else if (warp >= 8) {
    regs_dec<kTrWidenRegs>();
    // ============================================================ widening
    // Of lanes 32 q .. + 31 the warp has 16 keys of K (rows 16 half ..) and, of V^T, all dims of half of the columns
    // (n = 8 half .. + 7).  In pass i it widens K(i) and V(i - 1): S(i - 1), issued behind PV(i - 3), frees both.
    const int q = warp % 4, half = (warp - 8) / 4, g8 = lane / 4, t4 = lane % 4;
    const uint32_t lanes = static_cast<uint32_t>(32 * q) << 16;
    const uint32_t t_k = tmem + lanes + (static_cast<uint32_t>(16 * half) << 16) + G::kK;
    const uint32_t t_v = tmem + lanes + G::kVt + 32 * half;
    // K: rows g8 and g8 + 8 are keys in groups g8 / 2 and g8 / 2 + 4, d/4 codes each
    const int k_row = 4 * q + 2 * half + (g8 & 1);
    const int k_codes = g8 / 2 * G::kGroup + k_row * (D / 2) + t4 * (D / 8);
    const int k_scale = G::kKs + (16 * (g8 / 2) + k_row) * (D / 16) + t4 * (D / 64);
    // V: the matrix of columns n and n + 1 has the keys of all groups in one row; lane 4 r + x loads bytes 4 x .. of the
    // key in group r / 2 + 4 (r % 2), and the transposed matrix's columns 2 t + i are columns n + i of thread t
    const int v_codes = D == 128 ? G::kV + (g8 / 2 + 4 * (g8 % 2)) * G::kVGroup + 8 * half * (D / 2) + 16 * q + 4 * t4
                                 : G::kV + t4 * G::kVGroup + 8 * half * (D / 2) + 8 * q + g8;
    // scales of the warp's dims (one or two groups of 16) as pairs of keys: lane 8 x + y takes column 4 n + x,
    // n = 8 half + y: rows 2 (n / 2) and the next of group x + 4 (n % 2)
    const int v_scale = G::kVs + (16 * (lane / 8 + 4 * (lane % 2)) + 8 * half + lane % 8 / 2 * 2) * (D / 16) +
                        (D == 128 ? 2 * q : q);
    uint32_t(*const s_scale)[12] = ctl->scales[warp - 8];
    const uint32_t* const my_scale = s_scale[D == 128 ? g8 / 4 * 4 + t4 : t4];
    for (int i = 0;; ++i) {
      if (!wait(ctl->ring_full[i % G::kStages], i / G::kStages)) break;
      const bool end = ctl->flags[i % kTrFlags] < 0;
      if (i > 0 && !wait(ctl->s_full[(i - 1) & 1], (i - 1) >> 1)) break;
      tc_fence_after();
      if (!end) {
        const uint8_t* const st = s_ring + i % G::kStages * G::kStage;
        uint32_t w[2][4], sc[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const uint8_t* const codes = st + k_codes + e * 4 * G::kGroup;
          const uint8_t* const scale = st + k_scale + e * 64 * (D / 16);
          // (a value vector that is not a number makes its key's scores NaN)
          if constexpr (D == 128) {
            *reinterpret_cast<uint4*>(w[e]) = *reinterpret_cast<const uint4*>(codes);
            sc[e] = fma_f16x2(e4m3x2_to_f16x2(*reinterpret_cast<const uint16_t*>(scale + (G::kVs - G::kKs))), 0u,
                              e4m3x2_to_f16x2(*reinterpret_cast<const uint16_t*>(scale)));
          } else {
            *reinterpret_cast<uint2*>(w[e]) = *reinterpret_cast<const uint2*>(codes);
            sc[e] = fma_f16x2(e4m3x2_to_f16x2(scale[G::kVs - G::kKs]), 0u, e4m3x2_to_f16x2(*scale));
          }
        }
#pragma unroll
        for (int part = 0; part < D / 64; ++part) {
          uint32_t r[16];
#pragma unroll
          for (int x = 0; x < 2; ++x)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              uint32_t h[4];
              unpack_e2m1x8(w[e][2 * part + x], h);
#pragma unroll
              for (int y = 0; y < 4; ++y)
                r[2 * (4 * x + y) + e] = part ? mul_f16x2_hi(h[y], sc[e]) : mul_f16x2_lo(h[y], sc[e]);
            }
          tmem_st_16x128b_x8(t_k + (i & 1) * (D / 2) + part * 32, r);
        }
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&ctl->k_full[i & 1]));
      }
      if (i > 0) {
        const int t = i - 1, slot = t % G::kStages;
        const uint8_t* const st = s_ring + slot * G::kStage;
        // A value vector that is not a number (NaN scales) is zero: its key's scores are NaN, and rows that do not see
        // the key multiply it by zero.
        const uint8_t* const scale = st + v_scale;
        if constexpr (D == 128) {
          const uint32_t both = __byte_perm(*reinterpret_cast<const uint16_t*>(scale),
                                            *reinterpret_cast<const uint16_t*>(scale + D / 16), 0x5140);
          s_scale[lane / 8][lane % 8] = max_f16x2(e4m3x2_to_f16x2(static_cast<uint16_t>(both)), 0u);
          s_scale[4 + lane / 8][lane % 8] = max_f16x2(e4m3x2_to_f16x2(static_cast<uint16_t>(both >> 16)), 0u);
        } else {
          s_scale[lane / 8][lane % 8] =
              max_f16x2(e4m3x2_to_f16x2(static_cast<uint16_t>(scale[0] | scale[D / 16] << 8)), 0u);
        }
        __syncwarp();
        uint32_t sv[8], r0[16];
        *reinterpret_cast<uint4*>(sv) = *reinterpret_cast<const uint4*>(my_scale);
        *reinterpret_cast<uint4*>(sv + 4) = *reinterpret_cast<const uint4*>(my_scale + 4);
        const uint8_t* const p = st + v_codes;
        if constexpr (D == 128) {
          uint32_t r1[16];
#pragma unroll
          for (int n = 0; n < 8; n += 2) {
            const uint32_t xa = movmatrix_trans(*reinterpret_cast<const uint32_t*>(p + n * (D / 2)));
            const uint32_t xb = movmatrix_trans(*reinterpret_cast<const uint32_t*>(p + (n + 1) * (D / 2)));
            uint32_t even[4], odd[4];  // dims 0, 2 of column n, then of n + 1; dims 1, 3
            unpack_e2m1x8((xa & 0x0f0f0f0fu) | ((xb << 4) & 0xf0f0f0f0u), even);
            unpack_e2m1x8(((xa >> 4) & 0x0f0f0f0fu) | (xb & 0xf0f0f0f0u), odd);
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              r0[2 * (n + e)] = mul_f16x2(even[2 * e], sv[n + e]);
              r0[2 * (n + e) + 1] = mul_f16x2(odd[2 * e], sv[n + e]);
              r1[2 * (n + e)] = mul_f16x2(even[2 * e + 1], sv[n + e]);
              r1[2 * (n + e) + 1] = mul_f16x2(odd[2 * e + 1], sv[n + e]);
            }
          }
          tmem_st_16x128b_x8(t_v + (16u << 16) + (t & 1) * 64, r1);
        } else {
#pragma unroll
          for (int n = 0; n < 8; n += 4) {
            uint32_t x[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) x[e] = p[e / 2 % 2 * 4 * G::kVGroup + (n + e / 4 * 2 + e % 2) * (D / 2)];
            const uint32_t xa = x[0] | x[2] << 8 | x[4] << 16 | x[6] << 24, xb = x[1] | x[3] << 8 | x[5] << 16 | x[7] << 24;
            uint32_t even[4], odd[4];
            unpack_e2m1x8((xa & 0x0f0f0f0fu) | ((xb << 4) & 0xf0f0f0f0u), even);
            unpack_e2m1x8(((xa >> 4) & 0x0f0f0f0fu) | (xb & 0xf0f0f0f0u), odd);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              r0[2 * (n + e)] = mul_f16x2(even[e], sv[n + e]);
              r0[2 * (n + e) + 1] = mul_f16x2(odd[e], sv[n + e]);
            }
          }
        }
        tmem_st_16x128b_x8(t_v + (t & 1) * 64, r0);
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(smem_u32(&ctl->ring_empty[slot]));
          mbar_arrive(smem_u32(&ctl->v_full[t & 1]));
        }
      }
      if (end) break;
    }
  } else {
    regs_inc<kTrSoftmaxRegs>();
    // ============================================================ softmax, outputs
    constexpr int H = G::kHalf;
    const int g = warp / 4, q = warp % 4, m_row = 32 * q + lane, tid = threadIdx.x % 128;
    const int my_group = m_row % 8 / 2 + 4 * (m_row / 8 % 2);  // of 16 keys
    const int my_key = 16 * my_group + 2 * (m_row / 16) + (m_row & 1);
    const uint32_t lanes = static_cast<uint32_t>(32 * q) << 16;
    const uint32_t t_s = tmem + lanes + g * H, t_o = tmem + lanes + G::kO + g * H;
    float* const s_nm = ctl->nm + g * H;
    float* const s_alpha = ctl->alpha + g * H;
    const uint32_t p_row = smem_u32(s_p) + m_row * 128;
    const int bar = 1 + g;
    int t = 0, unit_no = 0;
    bool ok = true;
    // ---- the first unit's queries, eight rows a warp: there is nothing else to do yet (64 rows, 4096 keys: 3 % of the
    // time less than by one warp)
    if (warp < N / 8) {
      TreeRows<N>& rows = ctl->rows[0];
      const TreeSeg seg = tree_walk<N>(a, ctl).s;
      if (threadIdx.x == 0) rows.seg = seg;
      const RowPlace p = place(seg, 8 * warp + lane % 8);
      if (lane < 8) rows.out[8 * warp + lane] = p.out;
#pragma unroll
      for (int x = 0; x < 8; x += kRowsIt) fetch(0, 8 * warp + x, __shfl_sync(0xffffffffu, p.from, x + lane / kPieces));
      cp_async_commit();
#pragma unroll 1
      for (int y = 0; 32 * y < min(seg.req.queries, 32 * a.words); ++y) {
        const uint32_t bits = p.out >= 0 ? a.tree[static_cast<size_t>(p.token) * a.words + y] : 0u;
        uint32_t mine = 0u;  // bit e: row e sees node 32 y + lane
#pragma unroll
        for (int e = 0; e < 8; ++e) mine |= (__shfl_sync(0xffffffffu, bits, e) >> lane & 1u) << e;
        reinterpret_cast<uint8_t*>(rows.seen[32 * y + lane])[warp] = static_cast<uint8_t>(mine);
      }
      cp_async_wait<0>();
      __syncwarp();
      float here = row_most(0, 8 * warp + lane % 8, lane / 8, 4);
      here = fmaxf(here, __shfl_xor_sync(0xffffffffu, here, 8));
      here = fmaxf(here, __shfl_xor_sync(0xffffffffu, here, 16));
      if (lane < 8) rows.most[8 * warp + lane] = here;
      bar_wait(3, 4 * N);
      float most[N / 32];
#pragma unroll
      for (int x = 0; x < N / 32; ++x) most[x] = rows.most[x * 32 + lane];
      factors(rows, most);  // (every warp all of them)
      __syncwarp();
      convert(0, rows, 8 * warp + lane / kLanes, lane < 8 * kLanes);
      fence_proxy_async_smem();
      bar_wait(3, 4 * N);
      if (threadIdx.x == 0) mbar_arrive(smem_u32(&ctl->q_full[0]));
    }
    if (threadIdx.x == 0 && !a.whole_tiles) a.desc[blockIdx.x] = make_int4(-1, 0, 0, 0);
    // The four warps of a half meet at barriers that no time limit ends, so they leave together: a warp whose wait
    // has run out goes on to the next vote.
    for (int u = 0;; ++u) {
      ok = wait(ctl->q_full[u & 1], u >> 1);
      if (tid < H) s_nm[tid] = -kDecNone;
      if (bar_any(bar, 128, !ok)) break;
      const TreeRows<N>& rows = ctl->rows[u & 1];
      const int n = rows.seg.n;
      if (n == 0) break;
      bool leave = false;
      const float c = rows.c, lazy = rows.apart ? -INFINITY : kDecLazy;
      const int keys = rows.seg.req.keys, before = keys - rows.seg.req.queries, tile0 = rows.seg.tile;
      const int clean_tiles = before / kTrKeys - tile0;  // whose keys all rows see, if their pages are there
      float l[H], nm[H];
#pragma unroll
      for (int i = 0; i < H; ++i) {
        l[i] = 0.f;
        nm[i] = -kDecNone;
      }
#pragma unroll 1
      for (int j = 0; j < n; ++j, ++t) {
        ok = ok && wait(ctl->s_full[t & 1], t >> 1);
        tc_fence_after();
        const uint32_t t_here = t_s + (t & 1) * N;
        float x[H];
        auto scores = [&]() {
          uint32_t r[H];
          tmem_ld_cols<H>(t_here, r);
          tmem_ld_wait();
#pragma unroll
          for (int i = 0; i < H; ++i) x[i] = __uint_as_float(r[i]);
        };
        // bit i: row i of the half sees the thread's key
        uint32_t see = ~0u;
        const int flags = ctl->flags[t % kTrFlags];
        const bool clean = j < clean_tiles && flags == 0xff;
        if (!clean) {
          const int key = (tile0 + j) * kTrKeys + my_key, node = key - before;
          if (key >= keys || !(flags >> my_group & 1) || node >= 32 * a.words)
            see = 0u;
          else if (node >= 0)
            see = rows.seen[node][g * H / 32] >> (g * H % 32);
        }
        auto mask = [&]() {
          if (clean) return;
#pragma unroll
          for (int i = 0; i < H; ++i) x[i] = see >> i & 1u ? x[i] : -INFINITY;
        };
        // scores in units of the exponent, relative to the rows' references
        auto relative = [&]() {
#pragma unroll
          for (int i = 0; i < H; i += 2) {
            const float2 y = fma_f32x2(f32x2(x[i], x[i + 1]), f32x2(c, c), f32x2(nm[i], nm[i + 1]));
            x[i] = y.x;
            x[i + 1] = y.y;
          }
        };
#pragma unroll 1
        for (bool moved = false;; moved = true) {
          scores();
          relative();
          mask();
          float big = x[0];
#pragma unroll
          for (int i = 1; i + 1 < H; i += 2) big = max3f(big, x[i], x[i + 1]);
          big = fmaxf(big, x[H - 1]);
          if (moved || !bar_any(bar, 128, big > lazy || !ok)) break;
          // ---- some row's reference moves: maxima of all rows over the tile's keys
          if (rows.apart) {
#pragma unroll 1
            for (int i0 = 0; i0 < H; i0 += 8) {
              uint32_t r[8];
              tmem_ld_cols<8>(t_here + i0, r);
              tmem_ld_wait();
#pragma unroll
              for (int i = 0; i < 8; ++i)
                r[i] = __float_as_uint(__fmul_rn(__uint_as_float(r[i]), rows.row_c[g * H + i0 + i]));
              tmem_st_cols<8>(t_here + i0, r);
            }
            tmem_st_wait();
          }
#pragma unroll 1
          for (int i0 = 0; i0 < H; i0 += 8) {
            uint32_t r[8];
            tmem_ld_cols<8>(t_here + i0, r);
            tmem_ld_wait();
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const float v = warp_max(see >> (i0 + i) & 1u ? __uint_as_float(r[i]) * c : -INFINITY);
              if (lane == 0) ctl->top[q][g * H + i0 + i] = v;
            }
          }
          bar_wait(bar, 128);
          if (tid < H) {
            const int col = g * H + tid;
            float v = fmaxf(fmaxf(ctl->top[0][col], ctl->top[1][col]), fmaxf(ctl->top[2][col], ctl->top[3][col]));
            const float m = -s_nm[tid];
            v = fmaxf(v - kDecBelow, m);
            s_alpha[tid] = ex2_mufu(m - v);
            s_nm[tid] = -v;
          }
          if (j > 0 && ok) ok = wait(ctl->pv_done[(t - 1) & 1], (t - 1) >> 1);
          leave = bar_any(bar, 128, !ok);
          if (leave) break;
#pragma unroll
          for (int i = 0; i < H; ++i) nm[i] = s_nm[i];
          if (j > 0) {
            tc_fence_after();
            uint32_t r[H];
            tmem_ld_cols<H>(t_o, r);
            tmem_ld_wait();
#pragma unroll
            for (int i = 0; i < H; ++i) {
              const float f = s_alpha[i];
              r[i] = __float_as_uint(__uint_as_float(r[i]) * f);
              l[i] *= f;
            }
            tmem_st_cols<H>(t_o, r);
            tmem_st_wait();
          }
        }
        if (leave) break;
        const uint32_t dst = p_row + (t & 1) * G::kPBytes;
#pragma unroll
        for (int i = 0; i < H; i += 8) {
          uint32_t w[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int y = i + 2 * e;
            const float2 p = f32x2(ex2_mufu(x[y]), ex2_mufu(x[y + 1]));
            const float2 sum = add_f32x2(f32x2(l[y], l[y + 1]), p);
            l[y] = sum.x;
            l[y + 1] = sum.y;
            w[e] = pack_f16x2(p.x, p.y);
          }
          st_shared_v4(dst + (((g * H + i) / 8 ^ (m_row & 7)) << 4), w[0], w[1], w[2], w[3]);
        }
        fence_proxy_async_smem();
        tc_fence_before();  // S has been read (and O perhaps rescaled)
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&ctl->p_full[t & 1]));
      }
      if (leave) break;
      // ---- the rows' sums over all keys: lanes exchange halves until each holds a row's sum of its warp
#pragma unroll
      for (int o = H / 2; o >= 1; o /= 2) {
        const bool high = lane & o;
#pragma unroll
        for (int i = 0; i < o; ++i) {
          const float keep = high ? l[i + o] : l[i], send = high ? l[i] : l[i + o];
          l[i] = keep + __shfl_xor_sync(0xffffffffu, send, o);
        }
      }
#pragma unroll
      for (int o = H; o < 32; o *= 2) l[0] += __shfl_xor_sync(0xffffffffu, l[0], o);
      if (lane < H) ctl->top[q][g * H + lane] = l[0];
      if (bar_any(bar, 128, !ok)) break;
      const bool whole = n == rows.seg.tiles;
      const size_t slot = (2 * static_cast<size_t>(blockIdx.x) + (unit_no > 0 ? 1 : 0)) * N;
      if (tid < H) {
        const int col = g * H + tid;
        const float sum = (ctl->top[0][col] + ctl->top[1][col]) + (ctl->top[2][col] + ctl->top[3][col]);
        const float m = -s_nm[tid];
        const int at = rows.out[col];
        // nothing seen: O = 0 (a NaN sum stays NaN)
        s_alpha[tid] = sum == 0.f ? 0.f : a.v_descale / sum;
        if (at >= 0) {
          if (whole)
            a.lse[at] = sum == 0.f ? -INFINITY : m * kLn2F + logf(sum);
          else
            a.part_ml[slot + col] = make_float2(m, sum);
        }
      }
      if (threadIdx.x == 0 && rows.seg.tile == 0 && !whole) {
        // the unit begins here and ends in a later CTA: x is its last tile on the line (its first n end the share)
        const long long x = ctl->last - n + rows.seg.tiles - 1;
        const int row0 = rows.seg.block * N;
        a.desc[blockIdx.x] = merge_desc(rows.seg.req, rows.seg.head, row0, min(N, rows.seg.req.q_len * a.group - row0),
                                        2 * static_cast<int>(blockIdx.x) + (unit_no > 0 ? 1 : 0),
                                        share_of(ctl->total, n_cta, x) - static_cast<int>(blockIdx.x) + 1);
      }
      ok = wait(ctl->pv_done[(t - 1) & 1], (t - 1) >> 1);
      if (bar_any(bar, 128, !ok)) break;
      tc_fence_after();
      // ---- O: rows g8 and g8 + 8 of the 32 lanes, and the two 16 further on, are four neighbouring dims (two for
      // d = 64) of columns 4 n + t4
      const int g8 = lane / 4, t4 = lane % 4;
      constexpr int kDims = D / 32;
      uint32_t lo[H / 2], hi[D == 128 ? H / 2 : 1];
      tmem_ld_16x128b<H / 2>(t_o, lo);
      if constexpr (D == 128) tmem_ld_16x128b<H / 2>(t_o + (16u << 16), hi);
      tmem_ld_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&ctl->o_empty));
      const int dim = D / 4 * q + kDims * g8;
#pragma unroll
      for (int n4 = 0; n4 < H / 4; ++n4) {
        const int col = g * H + 4 * n4 + t4, at = rows.out[col];
        float y[4] = {__uint_as_float(lo[2 * n4]), __uint_as_float(lo[2 * n4 + 1]), 0.f, 0.f};
        if constexpr (D == 128) {
          y[2] = __uint_as_float(hi[2 * n4]);
          y[3] = __uint_as_float(hi[2 * n4 + 1]);
        }
        if (at < 0) continue;
        if (whole) {
          const float f = s_alpha[4 * n4 + t4];
          __nv_bfloat16* const to = a.o + static_cast<size_t>(at) * D + dim;
          if constexpr (D == 128)
            *reinterpret_cast<uint2*>(to) = make_uint2(pack_bf16x2(y[0] * f, y[1] * f), pack_bf16x2(y[2] * f, y[3] * f));
          else
            *reinterpret_cast<uint32_t*>(to) = pack_bf16x2(y[0] * f, y[1] * f);
        } else {
          float* const to = a.part_o + (slot + col) * D + dim;
          if constexpr (D == 128)
            *reinterpret_cast<float4*>(to) = make_float4(y[0], y[1], y[2], y[3]);
          else
            *reinterpret_cast<float2*>(to) = make_float2(y[0], y[1]);
        }
      }
      ++unit_no;
      bar_wait(bar, 128);  // the next unit writes s_alpha and s_nm
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&ctl->q_empty[u & 1]));
    }
  }

  __syncthreads();
  if (threadIdx.x == 0 && ctl->abort) atomicExch(a.status, kStatusTimeout);
  if (warp == kTrMmaWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

}  // namespace exattn
