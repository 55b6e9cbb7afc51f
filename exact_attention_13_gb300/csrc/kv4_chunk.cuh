// kv4_chunk.cuh -- attention of many query rows over the paged 4-bit cache (prompt chunks).
//
// The same operation as kv4_attn.cuh for units of 256 query rows (one key head of one request, rows
// ordered by token, then by head of the group).  With that many rows the two products, not the
// cache's bytes, are the floor, so they run on tcgen05: S_h = Q_h K^T and O_h += P_h V for two tiles
// h of 128 rows, accumulators and probabilities in tensor memory, one thread per row in the softmax.
// The cache is widened once per tile of 128 keys and serves both row tiles: f16 K and V tiles in a
// ring of shared-memory slots, in the 128-byte-swizzled layout that the MMA descriptors expect.
//
// Roles (544 threads, one CTA a SM):
//   warps 0-7    softmax of tile 0 / tile 1; also load the query rows (scaled by a power of two into
//                [1, 2), f16) and write O and the log-sum-exp
//   warps 8-11   widen the keys, 32 of a tile each: codes and scales from global memory to registers a
//                tile ahead, code * scale (exact) to the ring
//   warps 12-15  widen the values, likewise
//   warp  16     issues the MMAs:  S0(0) S1(0) | PV0(j) S0(j+1) PV1(j) S1(j+1) | ...
// TMEM: S_0 at columns 0-127, S_1 at 128-255 (P_h, f16, over S_h), O_0 at 256, O_1 at 384.
//
// A CTA takes an equal share of the line of all tiles, as in kv4_attn.cuh; a unit that crosses CTAs
// is merged from partial sums afterwards.  Units of one key head follow each other on the line, so
// CTAs that run together read the same keys from L2.
//
// Measured (2070 MHz).  One prompt of 65536 tokens, 8 heads over 1, d 128: 7.32 ms, 1202 TFLOP/s (0.62 of
// cuBLAS bf16); four chunks of up to 512 tokens behind 4096 to 8192 keys, 32 heads over 8: 129.5 us for
// 116 GFLOP, 897 TFLOP/s (0.46), 5 us of that the start, 18 the queries and outputs of the two or three
// shares of units a CTA has, and 10 the merge.  Units of at most 128 rows have one row tile: the other's
// warps and accumulators idle, and its chain S, softmax, P V, S runs alone (64 requests of 4096 keys with 36
// to 128 rows a key head: 231 to 238 us, their bytes take 47 to 50).  Within a unit a key tile takes about 3400 cycles, the MMAs of its two row
// tiles 2048 of them: S reads Q and K from shared memory at its full rate, beside which V is read and the
// next tiles are written, and S of a row tile waits for its own softmax (2100 cycles) and P V.
//
// Every mbarrier wait is bounded in time; one
// that runs out sets the CTA's abort flag and the status word, and all roles leave.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cstdint>

#include "fa_fwd_kernel.cuh"
#include "kv4_attn.cuh"

namespace exattn {

constexpr int kChThreads = 544;
constexpr int kChMmaWarp = 16;
constexpr int kChRows = 256;
constexpr int kChKeys = 128;
// 544 threads get 96 registers each at launch; the widening warpgroups give up what the softmax takes
// (the MMA warp, alone in its warpgroup, keeps its 96).  Four chunks of 512 tokens: 134.4 us with 136 and 56
// registers, 131.0 with 128 and 64, 128.9 with 120 and 72, 130.8 with 112 and 80 (a register or a few spilled each time).
constexpr int kChLaunchRegs = 96, kChSoftmaxRegs = 120, kChWidenRegs = 72;
static_assert(kChSoftmaxRegs + kChWidenRegs == 2 * kChLaunchRegs, "registers of the block at launch");

__device__ __forceinline__ uint32_t max_f16x2(uint32_t a, uint32_t b) {  // NaN: the other one
  uint32_t y;
  asm("max.f16x2 %0, %1, %2;" : "=r"(y) : "r"(a), "r"(b));
  return y;
}
__device__ __forceinline__ uint32_t fma_f16x2(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t y;
  asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(y) : "r"(a), "r"(b), "r"(c));
  return y;
}

template <int D>
struct ChunkGeo {
  static constexpr int kTileBytes = 128 * D * 2;          // 128 rows of f16, boxes of 64 columns
  static constexpr int kSlots = D == 128 ? 4 : 8;         // K and V tiles in flight
  static constexpr int kKSteps = D / 16;                  // MMAs of one S
  static constexpr uint32_t kIdescS = instr_desc(128, 128, 0, false, false);
  static constexpr uint32_t kIdescPV = instr_desc(128, D, 0, false, true);
  __host__ __device__ static constexpr int s_off(int kb) {
    return kb >= kKSteps ? 0 : ((kb * 32 / 128) * 128 * 128 + kb * 32 % 128) >> 4;
  }
  static constexpr int kPvStep = 16 * 128 >> 4;
};

template <bool B>
struct ChunkMasked {
  static constexpr bool value = B;
};

// One share of a unit: tiles [tile, tile + n) of its `tiles`.
struct ChunkSegment {
  int r, head, block, tile, n, tiles;
  ReqShape req;
};

// A warp's place on the line, in shared memory: registers are scarce in the loops.
struct ChunkWalk {
  ChunkSegment s;
  int blocks;
  long long left;  // tiles of the share from s.tile on
};

struct ChunkCtrl {
  uint64_t q_full[2], s_full[2], o_full[2], p_full[2][2];
  uint64_t kv_full[8], kv_empty[8];
  uint64_t drain;
  uint32_t tmem_base;
  int abort;
  long long sum[kChThreads / 32];
  long long total, first, last;
  ChunkSegment start;
  ChunkWalk walk[kChThreads / 32];
};

template <int D>
constexpr int chunk_smem_bytes() {
  return (2 + ChunkGeo<D>::kSlots) * ChunkGeo<D>::kTileBytes + static_cast<int>(sizeof(ChunkCtrl)) + 1024;
}

// Tiles that the 256 rows of a block need: up to the last key that its last row sees.
__device__ __forceinline__ int chunk_tiles(const Kv4Args& a, const ReqShape& s, int block) {
  int seen = s.keys;
  if (a.causal) {
    const int last_row = min(s.q_len * a.group, (block + 1) * kChRows) - 1;
    seen = max(0, s.keys - s.queries + last_row / a.group + 1);
  }
  return max(1, (min(seen, s.keys) - 1) / kChKeys + 1);
}

__device__ __forceinline__ int chunk_blocks(const Kv4Args& a, const ReqShape& s) {
  return (s.q_len * a.group + kChRows - 1) / kChRows;
}

// Every role walks the CTA's share of the line by itself, segment by segment (warp-collective).
__device__ __forceinline__ void walk_begin(const Kv4Args& a, ChunkWalk* w, const ChunkCtrl* ctl) {
  if (threadIdx.x % 32 == 0) {
    w->s = ctl->start;
    w->blocks = chunk_blocks(a, w->s.req);
    w->left = ctl->last - ctl->first;
    w->s.n = static_cast<int>(min(static_cast<long long>(w->s.tiles - w->s.tile), w->left));
  }
  __syncwarp();
}

// To the next segment; false at the end of the share.
__device__ __forceinline__ bool walk_next(const Kv4Args& a, ChunkWalk* w) {
  __syncwarp();
  if (threadIdx.x % 32 == 0) {
    w->left -= w->s.n;
    if (w->left > 0) {
      w->s.tile = 0;
      if (++w->s.block == w->blocks) {
        w->s.block = 0;
        if (++w->s.head == a.hk) {
          w->s.head = 0;
          do {
            ++w->s.r;
            w->s.req = kv4_request(a, w->s.r);
            w->blocks = chunk_blocks(a, w->s.req);
          } while (w->blocks == 0 && w->s.r + 1 < a.b);
        }
      }
      w->s.tiles = chunk_tiles(a, w->s.req, w->s.block);
      w->s.n = static_cast<int>(min(static_cast<long long>(w->s.tiles), w->left));
    }
  }
  __syncwarp();
  return w->left > 0;
}

// Rows of the segment's unit, from its first one.
__device__ __forceinline__ int walk_rows(const Kv4Args& a, const ChunkWalk* w) {
  return w->s.req.q_len * a.group - w->s.block * kChRows;
}

// The CTA's share [first, last) of the line of `total` tiles; fills ctl->start.  Returns the number
// of CTAs that have work.
__device__ __forceinline__ int chunk_my_range(const Kv4Args& a, ChunkCtrl* ctl, long long& total,
                                              long long& first, long long& last) {
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  ReqShape s{0, 0, 0, 0};
  long long per_head = 0;  // tiles of one key head of the thread's request
  auto lane_request = [&](int l) {
    return ReqShape{__shfl_sync(0xffffffffu, s.q0, l), __shfl_sync(0xffffffffu, s.q_len, l),
                    __shfl_sync(0xffffffffu, s.keys, l), __shfl_sync(0xffffffffu, s.queries, l)};
  };
  // A request a thread; those of many blocks (a block is 256 / group tokens) by the whole warp.
  auto cost = [&](int r) -> long long {
    constexpr int kAlone = 4;
    s = r < a.b ? kv4_request(a, r) : ReqShape{0, 0, 0, 0};
    const int blocks = chunk_blocks(a, s);
    per_head = 0;
    if (blocks <= kAlone)
      for (int b = 0; b < blocks; ++b) per_head += chunk_tiles(a, s, b);
    for (unsigned many = __ballot_sync(0xffffffffu, blocks > kAlone); many; many &= many - 1) {
      const int l = __ffs(many) - 1;
      const ReqShape x = lane_request(l);
      long long sum = 0;
      for (int b = lane; b < chunk_blocks(a, x); b += 32) sum += chunk_tiles(a, x, b);
#pragma unroll
      for (int o = 16; o; o /= 2) sum += __shfl_xor_sync(0xffffffffu, sum, o);
      if (lane == l) per_head = sum;
    }
    return per_head * a.hk;
  };
  auto scan = [&](long long x) {
#pragma unroll
    for (int o = 1; o < 32; o *= 2) {
      const long long y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    if (lane == 31) ctl->sum[warp] = x;
    __syncthreads();
    for (int w = 0; w < warp; ++w) x += ctl->sum[w];
    return x;
  };
  long long mine = 0, tiles = 0;
  for (int r0 = 0; r0 < a.b; r0 += kChThreads) mine += tiles = cost(r0 + threadIdx.x);
  long long inc = scan(mine);
  total = 0;
  for (int w = 0; w < kChThreads / 32; ++w) total += ctl->sum[w];
  const int n = static_cast<int>(min(static_cast<long long>(gridDim.x), total));
  if (static_cast<int>(blockIdx.x) >= n) return n;
  first = share_begin(total, n, blockIdx.x);
  last = share_begin(total, n, blockIdx.x + 1);
  long long base = 0;
  for (int r0 = 0; r0 < a.b; r0 += kChThreads) {
    long long all = total;
    if (a.b > kChThreads) {
      __syncthreads();
      tiles = cost(r0 + threadIdx.x);
      inc = scan(tiles) + base;
      all = base;
      for (int w = 0; w < kChThreads / 32; ++w) all += ctl->sum[w];
    }
    const unsigned here = __ballot_sync(0xffffffffu, first >= inc - tiles && first < inc);
    if (here) {
      const int l = __ffs(here) - 1;
      long long off = first - __shfl_sync(0xffffffffu, inc - tiles, l);
      const long long head_tiles = __shfl_sync(0xffffffffu, per_head, l);
      const ReqShape x = lane_request(l);
      const int head = static_cast<int>(off / head_tiles);
      off -= head * head_tiles;
      // the block that holds tile `off` of the head, 32 blocks at a time
      for (int b0 = 0;; b0 += 32) {
        const int own = b0 + lane < chunk_blocks(a, x) ? chunk_tiles(a, x, b0 + lane) : 0;
        long long upto = own;
#pragma unroll
        for (int o = 1; o < 32; o *= 2) {
          const long long y = __shfl_up_sync(0xffffffffu, upto, o);
          if (lane >= o) upto += y;
        }
        const unsigned past = __ballot_sync(0xffffffffu, off < upto);
        if (past) {
          if (lane == __ffs(past) - 1) {
            ChunkSegment& c = ctl->start;
            c.r = r0 + warp * 32 + l;
            c.req = x;
            c.head = head;
            c.block = b0 + lane;
            c.tile = static_cast<int>(off - (upto - own));
            c.tiles = own;
          }
          break;
        }
        off -= __shfl_sync(0xffffffffu, upto, 31);
        if (b0 > chunk_blocks(a, x)) break;  // (cannot be: off lies below the head's tiles)
      }
    }
    base = all;
    if (first < base) break;
  }
  __syncthreads();
  return n;
}

template <int D>
__global__ void __launch_bounds__(kChThreads, 1) kv4_chunk_kernel(const Kv4Args a) {
  using G = ChunkGeo<D>;
  extern __shared__ __align__(1024) uint8_t ch_smem[];
  uint8_t* const smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(ch_smem) + 1023) &
                                                   ~static_cast<uintptr_t>(1023));
  uint8_t* const s_q = smem;
  uint8_t* const s_ring = smem + 2 * G::kTileBytes;
  ChunkCtrl* const ctl = reinterpret_cast<ChunkCtrl*>(s_ring + G::kSlots * G::kTileBytes);
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;

  grid_launch_dependents();
  {
    long long total, first, last;
    const int n_cta = chunk_my_range(a, ctl, total, first, last);
    if (static_cast<int>(blockIdx.x) >= n_cta) {
      if (threadIdx.x == 0) a.desc[blockIdx.x] = make_int4(-1, 0, 0, 0);
      return;
    }
    if (threadIdx.x == 0) {
      ctl->total = total;
      ctl->first = first;
      ctl->last = last;
    }
  }
  if (warp == kChMmaWarp) {
    tmem_alloc(smem_u32(&ctl->tmem_base), 512);
    tmem_relinquish();
  }
  if (threadIdx.x == 0) {
    for (int h = 0; h < 2; ++h) {
      mbar_init(smem_u32(&ctl->q_full[h]), 4);   // one arrival per softmax warp of the tile
      mbar_init(smem_u32(&ctl->s_full[h]), 1);
      mbar_init(smem_u32(&ctl->o_full[h]), 1);
      for (int p = 0; p < 2; ++p) mbar_init(smem_u32(&ctl->p_full[h][p]), 4);
    }
    for (int i = 0; i < G::kSlots; ++i) {
      mbar_init(smem_u32(&ctl->kv_full[i]), 4);  // one arrival per widening warp
      mbar_init(smem_u32(&ctl->kv_empty[i]), 1);
    }
    mbar_init(smem_u32(&ctl->drain), 1);
    ctl->abort = 0;
    fence_mbar_init();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = ctl->tmem_base;
  int* const abort_flag = &ctl->abort;
  auto wait = [&](uint64_t& bar, uint32_t parity) -> bool {
    return __all_sync(0xffffffffu, wait_phase(smem_u32(&bar), parity & 1u, abort_flag, a.status));
  };

  if (warp == kChMmaWarp) {
    // ============================================================ MMA issuer
    ChunkWalk* const w = &ctl->walk[kChMmaWarp];
    walk_begin(a, w, ctl);
    int t = 0;  // K's number in the ring (V: t + 1)
    int steps[2] = {0, 0}, segs[2] = {0, 0};
    const uint64_t q_desc = smem_desc(smem_u32(s_q), 16, 1024, kSwizzle128B);
    const uint64_t k_desc = smem_desc(smem_u32(s_ring), 16, 1024, kSwizzle128B);
    const uint64_t v_desc = smem_desc(smem_u32(s_ring), 128 * 128, 1024, kSwizzle128B);
    constexpr uint64_t kTile16 = G::kTileBytes >> 4;
    bool ok = true;
    auto issue_s = [&](int h, int tk) {
      const uint64_t qd = q_desc + h * kTile16, kd = k_desc + (tk % G::kSlots) * kTile16;
      if (elect_one()) {
        mma_chain_ss_off<G::kKSteps, 0, G::s_off(1), G::s_off(2), G::s_off(3), G::s_off(4),
                         G::s_off(5), G::s_off(6), G::s_off(7)>(tmem + h * 128, G::kIdescS, 0u, qd, kd);
        tc_commit(smem_u32(&ctl->s_full[h]));
      }
      __syncwarp();
    };
    // P V of one key tile, then S of the next (which overwrites P): V, the next K and the first
    // part of P have mostly come, so one probe looks for all three
    auto step = [&](int h, bool begins, bool more) -> bool {
      const int tv = t + 1, tk = more ? t + 2 : t + 1;
      uint64_t &bv = ctl->kv_full[tv % G::kSlots], &bk = ctl->kv_full[tk % G::kSlots];
      if (!__all_sync(0xffffffffu,
                      mbar_try_wait3(smem_u32(&bv), (tv / G::kSlots) & 1, smem_u32(&bk), (tk / G::kSlots) & 1,
                                     smem_u32(&ctl->p_full[h][0]), steps[h] & 1)))
        if (!wait(bv, tv / G::kSlots) || !wait(bk, tk / G::kSlots) || !wait(ctl->p_full[h][0], steps[h])) return false;
      const uint64_t vd = v_desc + (tv % G::kSlots) * kTile16;
#pragma unroll
      for (int part = 0; part < 2; ++part) {
        if (part == 1 && !wait(ctl->p_full[h][1], steps[h])) return false;
        tc_fence_after();
        if (elect_one())
          mma_chain_ts_off<4, 0, G::kPvStep, 8, 16, 24, 32, 40, 48, 56>(
              tmem + 256 + h * 128, G::kIdescPV, begins && part == 0 ? 0u : 1u, tmem + h * 128 + part * 32,
              vd + part * 4 * G::kPvStep);
        __syncwarp();
      }
      ++steps[h];
      if (more) {
        issue_s(h, tk);
      } else {
        if (elect_one()) tc_commit(smem_u32(&ctl->o_full[h]));
        __syncwarp();
      }
      return true;
    };
    do {
      const bool two = walk_rows(a, w) > 128;
      const int n = w->s.n;
      ok = wait(ctl->q_full[0], segs[0]++);
      if (two) ok = ok && wait(ctl->q_full[1], segs[1]++);
      ok = ok && wait(ctl->kv_full[t % G::kSlots], t / G::kSlots);
      if (!ok) break;
      tc_fence_after();
      issue_s(0, t);
      if (two) issue_s(1, t);
#pragma unroll 1
      for (int i = 0; i < (two ? 2 * n : n) && ok; ++i) {  // one copy of the step's code
        const int h = two ? i & 1 : 0, j = two ? i >> 1 : i;
        ok = step(h, j == 0, j + 1 < n);
        if (h == (two ? 1 : 0)) t += 2;
      }
    } while (ok && walk_next(a, w));
    // nothing this warp issued may still run when the TMEM is released
    __syncwarp();
    if (elect_one()) tc_commit(smem_u32(&ctl->drain));
    const uint64_t t0 = globaltimer_ns();
    while (!mbar_try_wait(smem_u32(&ctl->drain), 0) && globaltimer_ns() - t0 < kWaitLimitNs) {
    }
  } else if (warp >= 8) {
    regs_dec<kChWidenRegs>();
    // ============================================================ widening the cache
    // The warp's 32 keys of a tile, or their values: a lane takes 32 codes (16 bytes, two scales) of
    // one row at a time, 4 (d = 128) or 2 lanes a row.
    constexpr int kLanes = D / 32, kRowsIt = 32 / kLanes, kIt = 32 / kRowsIt;
    constexpr int kCode = D / 2, kScale = D / 16;
    const bool values = warp >= 12;
    const int part = lane % kLanes, row_in = lane / kLanes, row_w = warp % 4 * 32;
    const int page_rows = 1 << a.page_shift;
    const int block_bytes = kv4_block_bytes(page_rows, D);
    const unsigned page_bytes = static_cast<unsigned>(block_bytes) * 2u * static_cast<unsigned>(a.hk);
    ChunkWalk* const w = &ctl->walk[warp];
    walk_begin(a, w, ctl);

    // Chunk g of a row (8 values, 16 bytes) lies at chunk g ^ (row % 8) of its 128-byte line.  Lanes of
    // the second half of a row take their codes' halves in the other order: else they would store
    // to the banks that the first half stores to.
    const int swap = part & 2 ? 8 : 0;
    const uint32_t scale_sel = part & 2 ? 0x1032u : 0x3210u;
    uint32_t store_at[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int g = (part * 4 + (i ^ (part & 2))) & 7;
      store_at[i] = smem_u32(s_ring) + (part / 2) * (128 * 128) + (row_w + row_in) * 128 + ((g ^ (row_in & 7)) << 4);
    }
    static_assert(kRowsIt % 8 == 0 && kIt % 2 == 0, "iterations keep the swizzle and a 16-key group");

    // ---- loads, a tile ahead; the page ids of the two 16-key groups come a tile before them
    int key = w->s.tile * kChKeys + row_w, tiles_left = w->s.n, keys = w->s.req.keys;
    const int* ids = a.table + static_cast<size_t>(w->s.r) * a.width;
    const uint8_t* head = a.cache + static_cast<size_t>(w->s.head) * 2 * block_bytes;
    int id[2];
    auto fetch_ids = [&]() {
      id[0] = key < keys ? *(ids + (key >> a.page_shift)) : -1;
      id[1] = id[0];
      if (a.page_shift == 4) id[1] = key + 16 < keys ? *(ids + (key >> 4) + 1) : -1;
    };
    uint2 c0[kIt], c1[kIt];
    uint16_t sc[kIt], sc_values[kIt];
    auto load = [&]() {
#pragma unroll
      for (int g = 0; g < 2; ++g) {
        const bool ok = static_cast<unsigned>(id[g]) < static_cast<unsigned>(a.pages);
        const int row = ((key + 16 * g) & (page_rows - 1)) + row_in;
        const uint8_t* k = head + static_cast<size_t>(ok ? static_cast<unsigned>(id[g]) : 0u) * page_bytes;
        const uint8_t* codes = k + (values ? block_bytes : 0) + row * kCode + part * 16;
        const uint8_t* scales = k + page_rows * kCode + row * kScale + part * 2;
#pragma unroll
        for (int x = 0; x < kIt / 2; ++x) {
          const int it = g * (kIt / 2) + x;
          c0[it] = c1[it] = make_uint2(0u, 0u);
          sc[it] = sc_values[it] = 0;
          if (ok) {  // (a page that is not there: zeros, and the scores are masked)
            c0[it] = *reinterpret_cast<const uint2*>(codes + x * kRowsIt * kCode + swap);
            c1[it] = *reinterpret_cast<const uint2*>(codes + x * kRowsIt * kCode + (swap ^ 8));
            sc[it] = *reinterpret_cast<const uint16_t*>(scales + x * kRowsIt * kScale + (values ? block_bytes : 0));
            if (!values) sc_values[it] = *reinterpret_cast<const uint16_t*>(scales + x * kRowsIt * kScale + block_bytes);
          }
        }
      }
    };
    // (test builds that inject a stall widen nothing: the first wait for a tile runs out)
    const long long tiles = EXATTN_INJECT_STALL ? 0 : ctl->last - ctl->first;
    fetch_ids();
    // One copy of the code for the first loads and the later ones: the roles' loops together have to
    // stay in the instruction cache (a second copy of loads and conversions cost 8 %).
#pragma unroll 1
    for (long long i = -1; i < tiles; ++i) {
      if (i >= 0) {
        const long long t = 2 * i + (values ? 1 : 0);
        const int slot = static_cast<int>(t % G::kSlots);
        if (t >= G::kSlots && !wait(ctl->kv_empty[slot], static_cast<uint32_t>(t / G::kSlots - 1))) break;
#pragma unroll
        for (int it = 0; it < kIt; ++it) {
          // A value vector that is not a number (NaN scales) makes its key's scores NaN and is zero
          // itself: rows that do not see the key multiply it by zero.  max takes NaN to its other
          // operand, 0; the values' scale times 0 is 0 or NaN.
          uint32_t scales = e4m3x2_to_f16x2(sc[it]);
          if (values)
            scales = max_f16x2(scales, 0u);
          else
            scales = fma_f16x2(e4m3x2_to_f16x2(sc_values[it]), 0u, scales);
          scales = __byte_perm(scales, 0u, scale_sel);
          const uint32_t word[4] = {c0[it].x, c0[it].y, c1[it].x, c1[it].y};
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            uint32_t h[4];
            unpack_e2m1x8(word[x], h);
#pragma unroll
            for (int e = 0; e < 4; ++e) h[e] = x & 2 ? mul_f16x2_hi(h[e], scales) : mul_f16x2_lo(h[e], scales);
            st_shared_v4(store_at[x] + slot * G::kTileBytes + it * kRowsIt * 128, h[0], h[1], h[2], h[3]);
          }
        }
        fence_proxy_async_smem();  // the MMAs read the tile through the async proxy
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&ctl->kv_full[slot]));
      }
      if (i + 1 < tiles) {
        load();
        if (--tiles_left > 0) {
          key += kChKeys;
        } else if (walk_next(a, w)) {
          key = w->s.tile * kChKeys + row_w;
          tiles_left = w->s.n;
          keys = w->s.req.keys;
          ids = a.table + static_cast<size_t>(w->s.r) * a.width;
          head = a.cache + static_cast<size_t>(w->s.head) * 2 * block_bytes;
        }
        if (i + 2 < tiles) fetch_ids();
      }
    }
  } else {
    regs_inc<kChSoftmaxRegs>();
    // ============================================================ softmax, queries, outputs
    const int h = warp / 4, r_tile = threadIdx.x % 128;
    const uint32_t lane_addr = static_cast<uint32_t>(warp % 4 * 32) << 16;
    const uint32_t t_s = tmem + lane_addr + h * 128, t_o = tmem + lane_addr + 256 + h * 128;
    ChunkWalk* const w = &ctl->walk[warp];
    walk_begin(a, w, ctl);
    int t = 0;  // K's number in the ring
    int step = 0, seg = 0, unit_no = 0;
    bool ok = true;
    if (threadIdx.x == 0) a.desc[blockIdx.x] = make_int4(-1, 0, 0, 0);
    do {
      const int n = w->s.n;
      const bool two = walk_rows(a, w) > 128;
      if (threadIdx.x == 0 && w->s.tile == 0 && n < w->s.tiles) {
        // the unit begins here and ends in a later CTA: x is its last tile on the line
        const long long x = ctl->last - w->left + w->s.tiles - 1, total = ctl->total;
        const int n_cta = static_cast<int>(min(static_cast<long long>(gridDim.x), total));
        a.desc[blockIdx.x] = merge_desc(w->s.req, w->s.head, w->s.block * kChRows, min(kChRows, walk_rows(a, w)),
                                        2 * static_cast<int>(blockIdx.x) + (unit_no > 0 ? 1 : 0),
                                        share_of(total, n_cta, x) - static_cast<int>(blockIdx.x) + 1);
      }
      if (h == 0 || two) {
        const bool frees = threadIdx.x % 128 == 0 && (h == 1 || !two);
        float c;   // factor of the row's scores
        int sees;  // keys that the row sees
        {
          const int row = h * 128 + r_tile, urow = w->s.block * kChRows + row;
          const bool live = row < walk_rows(a, w);
          const int qi = urow / a.group, qg = urow - qi * a.group;
          sees = w->s.req.keys;
          if (a.causal && live) sees = min(sees, max(0, sees - w->s.req.queries + qi + 1));
          // ---- the warp's 32 query rows, scaled into [1, 2): kRow lanes take 16 bytes each of a row
          constexpr int kRow = D / 8, kRowsIt = 32 / kRow;
          const long long mine = live ? static_cast<long long>(w->s.req.q0 + qi) * a.q_row +
                                            static_cast<long long>(w->s.head * a.group + qg) * a.q_head
                                      : -1;
          c = 0.f;
#pragma unroll 4
          for (int it = 0; it < 32 / kRowsIt; ++it) {
            const int r = it * kRowsIt + lane / kRow, piece = lane % kRow;
            const long long at = __shfl_sync(0xffffffffu, mine, r);
            uint4 raw = make_uint4(0u, 0u, 0u, 0u);
            if (at >= 0) raw = *(reinterpret_cast<const uint4*>(a.q + at) + piece);
            float f[8], amax = 0.f;
            unpack_bf16x8(raw, f);
#pragma unroll
            for (int e = 0; e < 8; e += 2) amax = max3f(amax, fabsf(f[e]), fabsf(f[e + 1]));
#pragma unroll
            for (int o = 1; o < kRow; o *= 2) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
            uint32_t ex = __float_as_uint(amax) >> 23;
            ex = ex == 255u ? 127u : min(max(ex, 1u), 253u);
            const float down = __uint_as_float((254u - ex) << 23), up = a.c * __uint_as_float(ex << 23);
            const float theirs = __shfl_sync(0xffffffffu, up, (lane & (kRowsIt - 1)) * kRow);
            if (lane / kRowsIt == it) c = theirs;  // the row of lane it * kRowsIt + ... is its own
            const int row_in = warp % 4 * 32 + r;
            st_shared_v4(smem_u32(s_q) + h * G::kTileBytes + row_in * 128 + (piece / 8) * (128 * 128) +
                             (((piece & 7) ^ (row_in & 7)) << 4),
                         pack_f16x2(f[0] * down, f[1] * down), pack_f16x2(f[2] * down, f[3] * down),
                         pack_f16x2(f[4] * down, f[5] * down), pack_f16x2(f[6] * down, f[7] * down));
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(smem_u32(&ctl->q_full[h]));
        }
        // pages of the segment that are not there: then every tile looks at its own page ids
        bool holes = false;
        {
          const int key_end = min(w->s.req.keys, (w->s.tile + n) * kChKeys);
          const int* ids = a.table + static_cast<size_t>(w->s.r) * a.width;
          for (int p = ((w->s.tile * kChKeys) >> a.page_shift) + lane; (p << a.page_shift) < key_end; p += 32)
            holes |= static_cast<unsigned>(*(ids + p)) >= static_cast<unsigned>(a.pages);
        }
        holes = __any_sync(0xffffffffu, holes);
        int lim = sees - w->s.tile * kChKeys;  // keys of the next tile that the row sees
        float m = kDecNone, l = 0.f;
#pragma unroll 1
        for (int j = 0; j < n; ++j, ++step, t += 2, lim -= kChKeys) {
          ok = wait(ctl->s_full[h], step);
          if (!ok) break;
          tc_fence_after();
          // The last tile's S is issued after both tiles' P V of the previous keys: slots go back
          if (frees) {
            mbar_arrive(smem_u32(&ctl->kv_empty[t % G::kSlots]));
            if (j > 0) mbar_arrive(smem_u32(&ctl->kv_empty[(t - 1) % G::kSlots]));
          }
          // Twice over the row's scores, 64 at a time: the maximum, then the probabilities.  (All 128
          // in registers as one unrolled body did not fit the instruction cache beside the other
          // roles'; 32 at a time: 134 us instead of 129; once over the scores, the reference moved
          // between the halves and P published at the end: 148; S of 64 keys in two buffers a row
          // tile, issued two steps ahead: 158, for Q is then read from shared memory twice as
          // often.)  Masked and not are two copies of the code: selects for a mask that mostly leaves
          // all cost a third of the instructions.
          const bool masked = holes || __any_sync(0xffffffffu, lim < kChKeys);
          // bit i: the row sees key i of 16-key group g
          auto seen16 = [&](int g) {
            const int here = lim - 16 * g;
            unsigned seen = here >= 16 ? 0xffffu : here <= 0 ? 0u : (1u << here) - 1u;
            if (holes) {
              const int key = (w->s.tile + j) * kChKeys + 16 * g;
              const int* ids = a.table + static_cast<size_t>(w->s.r) * a.width;
              if (key < w->s.req.keys &&
                  static_cast<unsigned>(*(ids + (key >> a.page_shift))) >= static_cast<unsigned>(a.pages))
                seen = 0u;
            }
            return seen;
          };
          auto scores = [&](auto with_mask, int half, float (&s)[64]) {
            uint32_t r[2][32];
            tmem_ld32(t_s + half * 64, r[0]);
            tmem_ld32(t_s + half * 64 + 32, r[1]);
            tmem_ld_wait();
#pragma unroll
            for (int i = 0; i < 64; ++i) s[i] = __uint_as_float(r[i / 32][i % 32]);
            if constexpr (with_mask.value) {
#pragma unroll
              for (int g = 0; g < 4; ++g) {
                const unsigned seen = seen16(4 * half + g);
#pragma unroll
                for (int i = 0; i < 16; ++i)
                  if (!(seen >> i & 1u)) s[16 * g + i] = -INFINITY;
              }
            }
          };
          auto maximum = [&](auto with_mask) {
            float mp[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll 1
            for (int half = 0; half < 2; ++half) {
              float s[64];
              scores(with_mask, half, s);
#pragma unroll
              for (int i = 0; i < 64; i += 2) mp[i / 2 % 4] = max3f(mp[i / 2 % 4], s[i], s[i + 1]);
            }
            return fmaxf(fmaxf(mp[0], mp[1]), fmaxf(mp[2], mp[3]));
          };
          float top = masked ? maximum(ChunkMasked<true>{}) : maximum(ChunkMasked<false>{});
          // the reference m: kDecBelow under the maximum, moved when that grew by 8 since
          top *= c;
          if (j == 0) {
            m = fmaxf(top - kDecBelow, m);
          } else if (__any_sync(0xffffffffu, top > m + kDecLazy)) {
            const float m_new = fmaxf(top - kDecBelow, m);
            const float alpha = ex2_mufu(m - m_new);
            uint32_t r[32];
#pragma unroll 1
            for (int cb = 0; cb < D / 32; ++cb) {
              tmem_ld32(t_o + cb * 32, r);
              tmem_ld_wait();
#pragma unroll
              for (int i = 0; i < 32; i += 2) {
                const float2 v = mul_f32x2(f32x2(__uint_as_float(r[i]), __uint_as_float(r[i + 1])), f32x2(alpha, alpha));
                r[i] = __float_as_uint(v.x);
                r[i + 1] = __float_as_uint(v.y);
              }
              tmem_st32(t_o + cb * 32, r);
            }
            l *= alpha;
            m = m_new;
          }
          // P = 2^(s c - m) in f16 over S (columns already read), published in two parts of 64 keys
          auto publish = [&](auto with_mask) {
            float2 sum[4] = {f32x2(0.f, 0.f), f32x2(0.f, 0.f), f32x2(0.f, 0.f), f32x2(0.f, 0.f)};
            const float2 c2 = f32x2(c, c), nm = f32x2(-m, -m);
#pragma unroll 1
            for (int half = 0; half < 2; ++half) {
              float s[64];
              scores(with_mask, half, s);
              uint32_t p[32];
#pragma unroll
              for (int i = 0; i < 32; ++i) {
                const float2 x = fma_f32x2(f32x2(s[2 * i], s[2 * i + 1]), c2, nm);
                float p0 = ex2_mufu(x.x), p1 = ex2_mufu(x.y);
                if constexpr (with_mask.value) {  // whatever c is
                  p0 = s[2 * i] == -INFINITY ? 0.f : p0;
                  p1 = s[2 * i + 1] == -INFINITY ? 0.f : p1;
                }
                sum[i % 4] = add_f32x2(sum[i % 4], f32x2(p0, p1));
                p[i] = pack_f16x2(p0, p1);
              }
              tmem_st32(t_s + 32 * half, p);
              tmem_st_wait();
              tc_fence_before();
              __syncwarp();
              if (lane == 0) mbar_arrive(smem_u32(&ctl->p_full[h][half]));
            }
            sum[0] = add_f32x2(add_f32x2(sum[0], sum[1]), add_f32x2(sum[2], sum[3]));
            return sum[0].x + sum[0].y;
          };
          l += masked ? publish(ChunkMasked<true>{}) : publish(ChunkMasked<false>{});
        }
        if (!ok) break;
        // ---- O and the log-sum-exp, or the unit's partial sums
        ok = wait(ctl->o_full[h], seg++);
        if (!ok) break;
        tc_fence_after();
        if (frees) mbar_arrive(smem_u32(&ctl->kv_empty[(t - 1) % G::kSlots]));
        const int row = h * 128 + r_tile, urow = w->s.block * kChRows + row;
        const bool live = row < walk_rows(a, w), whole = n == w->s.tiles;
        const int qi = urow / a.group, qg = urow - qi * a.group;
        const float inv = l == 0.f ? 0.f : a.v_descale / l;
        const size_t at = static_cast<size_t>(w->s.req.q0 + qi) * a.hq + w->s.head * a.group + qg;
        const size_t slot = (2 * static_cast<size_t>(blockIdx.x) + (unit_no > 0 ? 1 : 0)) * kChRows + row;
        // Through shared memory, 128 bytes of each row at a time (64 bf16 columns, or 32 of a partial
        // sum), so that whole lines go to memory; the buffer is where the warp's own query rows lay, which
        // no MMA reads any more.  (Each lane storing its own row cost 3.4 us a unit.)
        const uint32_t stage_row = smem_u32(s_q) + h * G::kTileBytes + r_tile * 128;
        const uint8_t* const stage = s_q + h * G::kTileBytes + warp % 4 * 4096;
        const long long out_at = !live ? -1 : static_cast<long long>(whole ? at : slot);
        const int cols = whole ? 64 : 32;
#pragma unroll 1
        for (int col = 0; col < D; col += cols) {
#pragma unroll 1
          for (int cb = 0; cb < cols; cb += 32) {
            uint32_t r[32];
            tmem_ld32(t_o + col + cb, r);
            tmem_ld_wait();
            if (whole) {
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                uint32_t p[4];
#pragma unroll
                for (int e = 0; e < 4; ++e)
                  p[e] = pack_bf16x2(__uint_as_float(r[8 * i + 2 * e]) * inv, __uint_as_float(r[8 * i + 2 * e + 1]) * inv);
                st_shared_v4(stage_row + (((cb / 8 + i) ^ (lane & 7)) << 4), p[0], p[1], p[2], p[3]);
              }
            } else {
#pragma unroll
              for (int i = 0; i < 8; ++i)
                st_shared_v4(stage_row + ((i ^ (lane & 7)) << 4), r[4 * i], r[4 * i + 1], r[4 * i + 2], r[4 * i + 3]);
            }
          }
          __syncwarp();
#pragma unroll 2
          for (int it = 0; it < 8; ++it) {  // four rows at a time, eight lanes a row
            const int r = it * 4 + lane / 8, piece = lane % 8;
            const long long to = __shfl_sync(0xffffffffu, out_at, r);
            const uint4 y = *reinterpret_cast<const uint4*>(stage + r * 128 + ((piece ^ (r & 7)) << 4));
            if (to >= 0) {
              if (whole)
                reinterpret_cast<uint4*>(a.o + to * D + col)[piece] = y;
              else
                reinterpret_cast<uint4*>(a.part_o + to * D + col)[piece] = y;
            }
          }
          __syncwarp();
        }
        if (live && whole) a.lse[at] = l == 0.f ? -INFINITY : m * kLn2F + logf(l);
        if (live && !whole) a.part_ml[slot] = make_float2(m, l);
        tc_fence_before();
      } else {
        t += 2 * n;
      }
      ++unit_no;
    } while (walk_next(a, w));
  }

  __syncthreads();
  if (warp == kChMmaWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

}  // namespace exattn
