// kv4_attn.cuh -- attention of a few query rows over the paged 4-bit cache (decode).
//
//     O_i = sum_j p_ij v_j,   p_ij = softmax_j(scale q_i . k_j),   LSE_i = log sum_j e^(scale q_i . k_j)
//
// over the keys j < len of the row's request (causal: j <= len - q_len + i, the new tokens being the
// last of the cache).  A row that sees no key gets O = 0 and LSE = -inf.
//
// What bounds it.  Each cached value is 4.5 bits and meets 8, 16 or 32 query rows (NT = 1, 2, 4 eights):
// the floor is the cache's bytes over HBM.  At 6.7 TB/s an SM has to widen about 41 values a clock, and its
// ALU and FMA pipes each start 64 lanes a clock, so conversions are counted in instructions per value
// (beside 8 rows; beside 16 and 32 the products and the latencies weigh more, see below):
//  * one cvt widens two e2m1 codes to f16 and one f16x2 multiply applies their scales (code * scale
//    is exact in f16), one instruction a value in all;
//  * the products run as mma.m16n8k16 with the CACHE as the 16-row operand, straight from the
//    registers that widened it: S^T = K Q^T and O^T = V^T P^T, queries in the 8-wide operand.  The
//    tensor core then does 8 NT products a value (8 queries as the 16-row operand: 16, half of them
//    padding).  tcgen05 takes its wide operand from shared or tensor memory only: each widened value
//    would be written and read there again, 4 bytes of on-chip traffic for each half byte of HBM;
//  * the contraction index of a product may be permuted freely, so each lane owns 16 or 32
//    neighbouring dims (K) or 16 dims of four tokens (V) and reads its codes with wide loads;
//  * V needs two TOKENS side by side in a register: nibbles of two tokens' words are interleaved
//    before they are widened, 4 logic instructions for 16 values;
//  * P^T leaves the S^T accumulators in the layout that movmatrix transposes into the operand's.
// Queries are scaled by a power of two per row into [1, 2) before they become f16, so the conversion
// keeps bf16's 8 bits down to 2^-17 of the row's largest value.  P is rounded to f16 (2^-11 of each
// probability at most, beside the 2^-8 of a bf16 output): against 64 bits outputs are as far off as with P in
// fp32 (1.7e-3 in norm either way), and single ones differ from those by a bf16 step.
//
// Split.  The work of all requests is one line of tiles (64 to 256 keys of one key head, for one
// block of query rows); CTA i of n takes the i-th n-th of it, so ragged lengths balance by themselves and a
// single long request fills the GPU.  In a tile each warp takes 16 to 64 keys, in its own ring of
// cp.async stages, with its own softmax state: warps meet only at the end of a unit (one key head of
// one block of rows).  A unit that crosses CTAs leaves partial sums (O, max, sum) in the workspace,
// which a second kernel merges in a fixed order.
//
// Measured (2070 MHz, calls following each other).  64 requests of 500 to 8192 keys, 32 heads over 8, d 128:
// 72 us, 284 MB at 3.9 TB/s; 64 of 4096 keys each 65 us, 303 MB at 4.7.  The slope over the length is
// 5.8 TB/s; what comes on top is fixed: 13 us beside equal lengths, 23 beside ragged ones, of it the start
// (lengths, page ids and the first tiles follow each other from memory), the units' begins and ends, and 3
// for the merge.  262144 keys of one request, 32 heads over 4: 37.7 us, 4.0 TB/s, 12 of it fixed.  Up to 15
// rows a key head, 24 heads over 8, 16 requests: 50 us, 145 MB at 2.9 TB/s.  64 requests of 4096 keys (floor
// 46 us): 66 us with 8 rows a key head, 91 with 16, 163 with 32 (NT = 4: 255 registers, some spilled).
// Beside 8 rows instructions start in 56 % of the cycles, beside 16 in 43 % (their registers leave two warps
// a scheduler); the rest is waits for the instructions' fixed latencies.  Not
// faster: loads to registers instead of the rings (100 us for the first case), four CTAs a SM, strips of
// 64 keys at d 128, three stages, prefetches of page ids or of whole L2 lines.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cstdint>

#include "kv4_cache.cuh"
#include "rope.cuh"
#include "sm103_ptx.cuh"

namespace exattn {

constexpr int kDecWarps = 4;
constexpr int kDecThreads = 32 * kDecWarps;
// 16-key groups of a strip, one warp's share of a tile: 32 keys at head dim 128, 64 at 64 (half the
// work a key), 16 beside the 128 accumulators of 32 rows at 128 (with 32 keys registers were spilled).
template <int D, int R>
__host__ __device__ constexpr int dec_groups() { return D == 64 ? 4 : R == 32 ? 1 : 2; }
template <int D, int R>
__host__ __device__ constexpr int dec_strip() { return 16 * dec_groups<D, R>(); }
template <int D, int R>
__host__ __device__ constexpr int dec_tile() { return kDecWarps * dec_strip<D, R>(); }
constexpr int kDecStages = 2;  // (3: no faster)
constexpr float kLn2F = 0.6931471805599453f;
// The reference m of a row's probabilities 2^(x - m) is set kDecBelow under the running maximum and
// O and l are rescaled only when the maximum has grown by more than 8 (log2) since: P then lies
// below 2^15, inside f16, keeps f16's full precision down to 2^-21 of the largest, and most strips
// skip the reduction over the warp.
constexpr float kDecBelow = 7.f;
constexpr float kDecLazy = kDecBelow + 8.f;
// m before a row has seen a key: finite, so that 2^(x - m) is 0 for a masked x = -inf and 2^(m - m') 0
constexpr float kDecNone = -3.0e38f;

struct Kv4Args {
  const __nv_bfloat16* q;  // [T, Hq, d], strides in elements
  long long q_row, q_head;
  const uint8_t* cache;
  const int* table;        // [B, width]
  const int* lens;         // [B]
  const int* q_offsets;    // [B + 1], or null: q_len rows each
  __nv_bfloat16* o;        // [T, Hq, d]
  float* lse;              // [T, Hq]
  float* part_o;           // [2 n][R][d]
  float2* part_ml;         // [2 n][R] (max, sum)
  int* status;             // device status word (kv4_chunk.cuh)
  int4* desc;              // [n] unit to merge (merge_desc), or x < 0
  long long q_len;
  int t, b, hq, hk, group, width, page_shift, pages;
  int causal;
  int whole_tiles;         // > 0: units are not split, each counts as this many tiles
  float c;                 // scale * log2(e) * key descale
  float v_descale;
  const uint32_t* tree;    // [T, words]: the nodes that a query sees among its request's (TREE)
  int words;
};

// A request's first row, its rows that there are, its keys, and its queries: more than the rows where its
// offsets reach past the end of q (a batch cut short).  The causal mask goes by the queries.
struct ReqShape {
  int q0, q_len, keys, queries;
};

__device__ __forceinline__ ReqShape kv4_request(const Kv4Args& a, int r) {
  ReqShape s;
  long long q0, q1;
  if (a.q_offsets) {
    q0 = *(a.q_offsets + r);
    q1 = *(a.q_offsets + r + 1);
  } else {
    q0 = a.q_len * r;
    q1 = q0 + a.q_len;
  }
  // offsets and lengths are device data: keep what they address inside the buffers
  s.q0 = static_cast<int>(min(max(q0, 0ll), static_cast<long long>(a.t)));
  q1 = max(q1, static_cast<long long>(s.q0));
  s.q_len = static_cast<int>(min(q1, static_cast<long long>(a.t))) - s.q0;
  s.queries = static_cast<int>(q1) - s.q0;
  const long long room = static_cast<long long>(a.width) << a.page_shift;
  s.keys = static_cast<int>(min(static_cast<long long>(max(*(a.lens + r), 0)), room));
  return s;
}

// Blocks of R query rows, and tiles of a unit (one block, one key head) of a request; a request
// without keys keeps one (empty) tile, so that its rows are written.
template <int R>
__device__ __forceinline__ int kv4_blocks(const Kv4Args& a, const ReqShape& s) {
  return static_cast<int>((static_cast<long long>(s.q_len) * a.group + R - 1) / R);
}
template <int D, int R>
__device__ __forceinline__ int kv4_tiles(const ReqShape& s) {
  return max(1, (s.keys - 1) / dec_tile<D, R>() + 1);
}

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, uint32_t bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes)
               : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b) {
  uint32_t y;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(y) : "r"(a), "r"(b));
  return y;
}
// Both halves of a times the low (high) half of s.
__device__ __forceinline__ uint32_t mul_f16x2_lo(uint32_t a, uint32_t s) {
  const __half2 y = __hmul2(*reinterpret_cast<const __half2*>(&a),
                            __low2half2(*reinterpret_cast<const __half2*>(&s)));
  return *reinterpret_cast<const uint32_t*>(&y);
}
__device__ __forceinline__ uint32_t mul_f16x2_hi(uint32_t a, uint32_t s) {
  const __half2 y = __hmul2(*reinterpret_cast<const __half2*>(&a),
                            __high2half2(*reinterpret_cast<const __half2*>(&s)));
  return *reinterpret_cast<const uint32_t*>(&y);
}
// Whether either half is NaN.
__device__ __forceinline__ bool any_nan_f16x2(uint32_t x) {
  const __half2 h = *reinterpret_cast<const __half2*>(&x);
  return !__hbeq2(h, h);
}
__device__ __forceinline__ uint32_t movmatrix_trans(uint32_t x) {
  uint32_t y;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
__device__ __forceinline__ void mma_16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                          uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Row k of a 16-key group's product operands is key (k & 8) | kv4_perm(k & 7): neighbouring lanes
// then read rows of both parities, which halves the bank conflicts of V's loads.
__device__ __forceinline__ int kv4_perm(int r) { return r ^ ((r >> 1) & 1); }

// Where the CTA's line of tiles runs: request, block of query rows, key head, tile (the unit's
// number within its request is block * hk + head).
struct TileCursor {
  int r, block, head, tile, blocks, tiles;
  ReqShape req;
};

// The line of `total` tiles in n equal shares (n <= total), the first total % n one longer: where
// share i begins, and the share that holds tile x.
__device__ __forceinline__ long long share_begin(long long total, int n, int i) {
  if (total <= 0x7fffffffll) {  // 64-bit divisions take about 100 instructions
    const unsigned t = static_cast<unsigned>(total), q = t / n, more = t - q * n;
    return q * i + min(more, static_cast<unsigned>(i));
  }
  return total / n * i + min(total % n, static_cast<long long>(i));
}
__device__ __forceinline__ int share_of(long long total, int n, long long x) {
  if (total <= 0x7fffffffll) {
    const unsigned t = static_cast<unsigned>(total), q = t / n, more = t - q * n;
    const unsigned y = static_cast<unsigned>(x), longer = more * (q + 1);
    return static_cast<int>(y < longer ? y / (q + 1) : more + (y - longer) / q);
  }
  const long long q = total / n, more = total % n, longer = more * (q + 1);
  return static_cast<int>(x < longer ? x / (q + 1) : more + (x - longer) / q);
}

// A unit to be merged: its first partial sum's slot and the number of parts, its first query token, its
// first row, its key head and its rows (<= 256).
__device__ __forceinline__ int4 merge_desc(const ReqShape& req, int head, int row0, int rows, int slot,
                                           int parts) {
  return make_int4(slot | parts << 16, req.q0, row0, head | rows << 16);
}

// To the next tile; true when the next unit begins with it.
template <int D, int R>
__device__ __forceinline__ bool cursor_next(const Kv4Args& a, TileCursor& c) {
  if (++c.tile < c.tiles) return false;
  c.tile = 0;
  if (++c.head < a.hk) return true;
  c.head = 0;
  if (++c.block < c.blocks) return true;
  c.block = 0;
  while (++c.r < a.b) {
    const ReqShape s = kv4_request(a, c.r);
    c.blocks = kv4_blocks<R>(a, s);
    c.tiles = a.whole_tiles ? a.whole_tiles : kv4_tiles<D, R>(s);
    c.req = s;
    if (c.blocks > 0) break;
  }
  return true;
}

// The CTA's range [first, last) of the line of `total` tiles, and the cursor at its first tile.
// Returns the number of CTAs that have work.
template <int D, int R>
__device__ __forceinline__ int kv4_my_range(const Kv4Args& a, long long* s_sum, TileCursor* s_cur,
                                            long long& total, long long& first, long long& last) {
  const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32;
  TileCursor c;
  auto cost = [&](int r) -> long long {
    c = TileCursor{r, 0, 0, 0, 0, 1, {0, 0, 0, 0}};
    if (r >= a.b) return 0;
    const ReqShape s = kv4_request(a, r);
    c.blocks = kv4_blocks<R>(a, s);
    c.tiles = a.whole_tiles ? a.whole_tiles : kv4_tiles<D, R>(s);
    c.req = s;
    return static_cast<long long>(c.blocks) * a.hk * c.tiles;
  };
  // inclusive scan over the block; s_sum keeps the warps' sums until the next barrier
  auto scan = [&](long long x) {
#pragma unroll
    for (int o = 1; o < 32; o *= 2) {
      const long long y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    if (lane == 31) s_sum[warp] = x;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kDecWarps; ++w)
      if (w < warp) x += s_sum[w];
    return x;
  };
  long long mine = 0, tiles = 0;
  for (int r = tid; r < a.b; r += kDecThreads) mine += tiles = cost(r);
  long long inc = scan(mine);
  total = 0;
#pragma unroll
  for (int w = 0; w < kDecWarps; ++w) total += s_sum[w];
  const long long piece = a.whole_tiles ? a.whole_tiles : 1;  // shares are whole pieces
  const long long pieces = a.whole_tiles ? total / piece : total;
  const int n = static_cast<int>(min(static_cast<long long>(gridDim.x), pieces));
  if (static_cast<int>(blockIdx.x) >= n) return n;
  first = share_begin(pieces, n, blockIdx.x) * piece;
  last = share_begin(pieces, n, blockIdx.x + 1) * piece;
  // up to one request a thread, the scan above is the line itself; else it is redone in pieces
  long long base = 0;
  for (int r0 = 0; r0 < a.b; r0 += kDecThreads) {
    long long all = total;
    if (a.b > kDecThreads) {
      __syncthreads();
      tiles = cost(r0 + tid);
      inc = scan(tiles) + base;
      all = base;
#pragma unroll
      for (int w = 0; w < kDecWarps; ++w) all += s_sum[w];
    }
    const long long lo = inc - tiles;
    if (first >= lo && first < inc) {
      const long long off = first - lo;
      const int u = off <= 0x7fffffffll ? static_cast<int>(off) / c.tiles : static_cast<int>(off / c.tiles);
      c.tile = static_cast<int>(off - static_cast<long long>(u) * c.tiles);
      c.block = u / a.hk;
      c.head = u - c.block * a.hk;
      *s_cur = c;
    }
    base = all;
    if (first < base) break;
  }
  __syncthreads();
  return n;
}

template <int D, int R>
__host__ __device__ constexpr int dec_strip_bytes() { return dec_strip<D, R>() * (D + D / 8); }

template <int D, int NT>
__host__ __device__ constexpr int dec_smem_bytes() {
  return kDecWarps * kDecStages * dec_strip_bytes<D, 8 * NT>() + kDecWarps * (D / 16) * NT * 32 * 16 +
         NT * (D / 32) * 32 * 16;
}

// TREE: requests' last keys are the nodes of a tree, of which each row sees those of its bits; only tiles with such keys
// look at bits (64 requests of 4096 keys, 8 rows a key head: 67.1 us, causal 66; 16 rows: 91.3).
template <int D, int NT, bool TREE = false>
__global__ void __launch_bounds__(kDecThreads, NT == 1 ? 3 : 2) kv4_decode_kernel(const Kv4Args a) {
  constexpr int R = 8 * NT;            // query rows of a unit
  constexpr int MT = D / 16;           // 16-dim tiles of O^T
  constexpr int QW = D / 8;            // f16x2 words of one lane's share of a query row
  constexpr int KW = D / 32;           // code words of a lane's share of a key
  constexpr int VW = D / 64;           // code words of a lane's share of a value
  constexpr int kCode = D / 2, kScale = D / 16;  // bytes of a row's codes and scales
  constexpr int TG = dec_groups<D, R>(), kStrip = dec_strip<D, R>();
  constexpr int kKs = kStrip * kCode, kV = kKs + kStrip * kScale, kVs = kV + kKs;
  constexpr unsigned kAll = (1u << TG) - 1;
  extern __shared__ __align__(128) uint8_t dec_smem[];
  __shared__ long long s_sum[kDecWarps];
  __shared__ TileCursor s_cur;
  __shared__ float s_m[kDecWarps][R], s_l[kDecWarps][R];
  __shared__ __align__(8) float s_c[R];  // factors of the rows' scores

  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  const int g8 = lane / 4, t4 = lane % 4;
  uint8_t* const ring = dec_smem + warp * (kDecStages * dec_strip_bytes<D, R>());
  // the warps' sums at the end of a unit, and its queries as the products' operand
  float4* const area = reinterpret_cast<float4*>(dec_smem + kDecWarps * kDecStages * dec_strip_bytes<D, R>());
  uint4* const s_q = reinterpret_cast<uint4*>(area + kDecWarps * MT * NT * 32);  // [nt][w][lane]

  grid_launch_dependents();
  long long total, first, last;
  const int n_cta = kv4_my_range<D, R>(a, s_sum, &s_cur, total, first, last);
  if (static_cast<int>(blockIdx.x) >= n_cta) {
    if (threadIdx.x == 0 && !a.whole_tiles) a.desc[blockIdx.x] = make_int4(-1, 0, 0, 0);
    return;
  }
  const int steps = static_cast<int>(last - first);
  TileCursor cur = s_cur, ld = s_cur;
  const int page_rows = 1 << a.page_shift;
  const int block_bytes = kv4_block_bytes(page_rows, D);

  // ---- loads: the strip's 16-key groups, one page id each, fetched a step ahead
  const unsigned page_bytes = static_cast<unsigned>(block_bytes) * 2u * static_cast<unsigned>(a.hk);
  constexpr int kPer = 16 * kCode / 512;  // 16-byte copies of a lane for one group's codes
  // the lane's copy of the strip's scales: kScale copies for each of (K, V) x groups, 32 or 16 in all
  static_assert(2 * TG * kScale <= 32, "at most one copy of scales a lane");
  const int sc_group = lane / kScale % TG, sc_kv = lane / (kScale * TG) & 1;
  const int sc_dst = (sc_kv ? kVs : kKs) + sc_group * 16 * kScale + (lane % kScale) * 16;
  const uint32_t ring_u32 = smem_u32(ring);
  const uint8_t *code_base, *scale_base;  // of the head, with the lane's offset
  const int* row_ids;                     // the request's row of the table
  auto set_head = [&]() {
    const uint8_t* h = a.cache + static_cast<size_t>(ld.head) * 2 * block_bytes;
    code_base = h + lane * 16;
    scale_base = h + (sc_kv ? block_bytes : 0) + static_cast<size_t>(page_rows) * kCode + (lane % kScale) * 16;
    row_ids = a.table + static_cast<size_t>(ld.r) * a.width;
  };
  // Brings a unit's query rows into L1 ahead of their use: the loads' results are not wanted.
  auto touch_queries = [&]() {
    constexpr int kLines = D * 2 / 128;
#pragma unroll
    for (int x = 0; x < (R * kLines + 31) / 32; ++x) {
      const int line = x * 32 + lane, row = ld.block * R + line / kLines;
      if (line < R * kLines && row < ld.req.q_len * a.group) {
        const int qi = row / a.group, qg = row - qi * a.group;
        const __nv_bfloat16* p = a.q + static_cast<long long>(ld.req.q0 + qi) * a.q_row +
                                 static_cast<long long>(ld.head * a.group + qg) * a.q_head + line % kLines * 64;
        uint32_t unused;
        asm volatile("ld.global.b32 %0, [%1];" : "=r"(unused) : "l"(p));
      }
    }
  };
  int id[TG];
  int ld_left = steps;
  unsigned seen = 0;  // TG bits a strip in flight: the group's page exists
  auto fetch_ids = [&]() {
    const int key0 = ld.tile * dec_tile<D, R>() + warp * kStrip;
#pragma unroll
    for (int g = 0; g < TG; ++g) {
      const int key = key0 + 16 * g;
      // groups that share a page share its id
      if (g > 0 && (key & (page_rows - 1)) != 0) id[g] = id[g - 1];
      else id[g] = key < ld.req.keys ? *(row_ids + (key >> a.page_shift)) : -1;
    }
  };
  auto issue = [&](int stage) {
    seen <<= TG;
    if (ld_left > 0) {
      const uint32_t dst = ring_u32 + stage * dec_strip_bytes<D, R>();
      const int key0 = ld.tile * dec_tile<D, R>() + warp * kStrip;
      uint32_t sc_n = 0;
      size_t sc_at = 0;
#pragma unroll
      for (int g = 0; g < TG; ++g) {
        const bool ok = static_cast<unsigned>(id[g]) < static_cast<unsigned>(a.pages);
        // a page that is not there: copies of zero bytes, which write zeros and read nothing
        const uint32_t n = ok ? 16u : 0u;
        const size_t at = static_cast<size_t>(ok ? static_cast<unsigned>(id[g]) : 0u) * page_bytes;
        const int row = (key0 + 16 * g) & (page_rows - 1);
        const uint8_t* k = code_base + at + row * kCode;
        const uint8_t* v = k + block_bytes;
        const uint32_t to = dst + g * 16 * kCode + lane * 16;
#pragma unroll
        for (int p = 0; p < kPer; ++p) {
          cp_async16(to + p * 512, k + p * 512, n);
          cp_async16(to + kV + p * 512, v + p * 512, n);
        }
        if (sc_group == g) {
          sc_n = n;
          sc_at = at + row * kScale;
        }
        seen |= (ok ? 1u : 0u) << g;
      }
      if (2 * TG * kScale == 32 || lane < 2 * TG * kScale) cp_async16(dst + sc_dst, scale_base + sc_at, sc_n);
      if (--ld_left > 0) {
        if (cursor_next<D, R>(a, ld)) {
          set_head();
          touch_queries();
        }
        fetch_ids();
      }
    }
    cp_async_commit();
  };

  set_head();
  fetch_ids();
  touch_queries();
#pragma unroll
  for (int s = 0; s < kDecStages; ++s) issue(s);

  // ---- state of the unit at hand
  int min_lim = 0, max_lim = 0;  // fewest and most keys that a row of the unit sees
  float m[NT][2], l[NT][2], o[MT][NT][4];
  bool fresh = true, whole_start = cur.tile == 0;
  int unit_no = 0;
  int4 merge = make_int4(-1, 0, 0, 0);

  int stage = 0;
  // keys that row `row` of the unit sees, one behind the other (a padding row: all; of a tree those before it)
  auto row_keys = [&](int row) {
    const int at = cur.block * R + row;
    if constexpr (TREE) return at < cur.req.q_len * a.group ? max(0, cur.req.keys - cur.req.queries) : cur.req.keys;
    const int behind = a.causal && at < cur.req.q_len * a.group ? cur.req.queries - at / a.group - 1 : 0;
    return max(0, cur.req.keys - behind);
  };
  for (int step = 0; step < steps; ++step) {
    if (fresh) {
      fresh = false;
      const ReqShape req = cur.req;
      const int head = cur.head, row0 = cur.block * R, rows = req.q_len * a.group;
      // Warp nt turns eight rows into the operand for all warps: held in registers by each warp they
      // would cost 16 registers (of 128) per eight rows, and four conversions.
      if (warp < NT) {
        const int row = row0 + warp * 8 + g8;
        uint4 raw[QW / 4];
        const bool live = row < rows;
        const int qi = row / a.group, qg = row - qi * a.group;
        const __nv_bfloat16* src = a.q + static_cast<long long>(req.q0 + qi) * a.q_row +
                                   static_cast<long long>(head * a.group + qg) * a.q_head + t4 * (D / 4);
        float amax = 0.f;
#pragma unroll
        for (int w = 0; w < QW / 4; ++w) {
          raw[w] = live ? *(reinterpret_cast<const uint4*>(src) + w) : make_uint4(0u, 0u, 0u, 0u);
          float f[8];
          unpack_bf16x8(raw[w], f);
#pragma unroll
          for (int e = 0; e < 8; ++e) amax = fmaxf(amax, fabsf(f[e]));
        }
        amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
        amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
        // power of two that brings the row's largest value into [1, 2) (below 4 at the top end);
        // an infinite or NaN row is left as it is
        uint32_t ex = __float_as_uint(amax) >> 23;
        ex = ex == 255u ? 127u : min(max(ex, 1u), 253u);
        const float down = __uint_as_float((254u - ex) << 23);
#pragma unroll
        for (int w = 0; w < QW / 4; ++w) {
          float f[8];
          unpack_bf16x8(raw[w], f);
          s_q[(warp * (QW / 4) + w) * 32 + lane] =
              make_uint4(pack_f16x2(f[0] * down, f[1] * down), pack_f16x2(f[2] * down, f[3] * down),
                         pack_f16x2(f[4] * down, f[5] * down), pack_f16x2(f[6] * down, f[7] * down));
        }
        if (t4 == 0) s_c[warp * 8 + g8] = a.c * __uint_as_float(ex << 23);
      }
      __syncthreads();
      min_lim = 0x7fffffff;
      max_lim = 0;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
        for (int cc = 0; cc < 2; ++cc) {
          const int row = nt * 8 + 2 * t4 + cc, k = row_keys(row);
          min_lim = min(min_lim, k);
          if (row0 + row < rows) max_lim = max(max_lim, TREE ? req.keys : k);
          m[nt][cc] = kDecNone;
          l[nt][cc] = 0.f;
        }
      }
#pragma unroll
      for (int x = 1; x <= 2; x *= 2) {
        min_lim = min(min_lim, __shfl_xor_sync(0xffffffffu, min_lim, x));
        max_lim = max(max_lim, __shfl_xor_sync(0xffffffffu, max_lim, x));
      }
#pragma unroll
      for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 4; ++e) o[i][nt][e] = 0.f;
    }

    cp_async_wait<kDecStages - 1>();
    __syncwarp();
    const int key0 = cur.tile * dec_tile<D, R>() + warp * kStrip;
    const unsigned have = (seen >> (TG * (kDecStages - 1))) & kAll;
    if (key0 < max_lim && have) {
      const uint8_t* const st = ring + stage * dec_strip_bytes<D, R>();
      const bool full = key0 + kStrip <= min_lim && have == kAll;
      float x[TG][NT][4];
      // ---- S^T = K Q^T
#pragma unroll
      for (int tg = 0; tg < TG; ++tg) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 4; ++e) x[tg][nt][e] = 0.f;
        const int k0 = tg * 16 + kv4_perm(g8), k1 = k0 + 8;
        uint32_t w0[KW], w1[KW];
        uint32_t sc0, sc1;  // scales of the lane's first and second 16 dims
        if constexpr (D == 128) {
          *reinterpret_cast<uint4*>(w0) = *reinterpret_cast<const uint4*>(st + k0 * kCode + t4 * 16);
          *reinterpret_cast<uint4*>(w1) = *reinterpret_cast<const uint4*>(st + k1 * kCode + t4 * 16);
          sc0 = e4m3x2_to_f16x2(*reinterpret_cast<const uint16_t*>(st + kKs + k0 * kScale + t4 * 2));
          sc1 = e4m3x2_to_f16x2(*reinterpret_cast<const uint16_t*>(st + kKs + k1 * kScale + t4 * 2));
        } else {
          *reinterpret_cast<uint2*>(w0) = *reinterpret_cast<const uint2*>(st + k0 * kCode + t4 * 8);
          *reinterpret_cast<uint2*>(w1) = *reinterpret_cast<const uint2*>(st + k1 * kCode + t4 * 8);
          sc0 = e4m3x2_to_f16x2(st[kKs + k0 * kScale + t4]);
          sc1 = e4m3x2_to_f16x2(st[kKs + k1 * kScale + t4]);
        }
#pragma unroll
        for (int w = 0; w < KW; ++w) {
          uint32_t h0[4], h1[4];
          unpack_e2m1x8(w0[w], h0);
          unpack_e2m1x8(w1[w], h1);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            h0[e] = w / 2 ? mul_f16x2_hi(h0[e], sc0) : mul_f16x2_lo(h0[e], sc0);
            h1[e] = w / 2 ? mul_f16x2_hi(h1[e], sc1) : mul_f16x2_lo(h1[e], sc1);
          }
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            const uint4 q = s_q[(nt * KW + w) * 32 + lane];
            mma_16816(x[tg][nt], h0[0], h1[0], h0[1], h1[1], q.x, q.y);
            mma_16816(x[tg][nt], h0[2], h1[2], h0[3], h1[3], q.z, q.w);
          }
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 4; e += 2) {
            const float2 y = mul_f32x2(f32x2(x[tg][nt][e], x[tg][nt][e + 1]),
                                       *reinterpret_cast<const float2*>(&s_c[nt * 8 + 2 * t4]));
            x[tg][nt][e] = y.x;
            x[tg][nt][e + 1] = y.y;
          }
      }

      // ---- V scales of the lane's tokens (two pairs a group)
      uint32_t vs[TG][2], b[TG][4];
#pragma unroll
      for (int tg = 0; tg < TG; ++tg)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int tok = tg * 16 + kv4_perm(2 * t4 + (e & 1)) + 8 * (e >> 1);
          b[tg][e] = st[kVs + tok * kScale + (D == 128 ? g8 : g8 / 2)];
        }
      if (!full) {
        // keys past the end and on missing pages must not meet P's zeros with a NaN scale
#pragma unroll
        for (int tg = 0; tg < TG; ++tg)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int tok = tg * 16 + kv4_perm(2 * t4 + (e & 1)) + 8 * (e >> 1);
            if (key0 + tok >= cur.req.keys || !((have >> tg) & 1u)) b[tg][e] = 0u;
          }
      }
#pragma unroll
      for (int tg = 0; tg < TG; ++tg)
#pragma unroll
        for (int pr = 0; pr < 2; ++pr)
          vs[tg][pr] = e4m3x2_to_f16x2(static_cast<uint16_t>(b[tg][2 * pr] | (b[tg][2 * pr + 1] << 8)));
      // A value vector that is not a number makes the rows that see its key NaN through their
      // scores; its scales become zero, because rows that do not see it multiply it by zero.
      uint32_t sum_vs = hadd_f16x2(vs[0][0], vs[0][1]);
#pragma unroll
      for (int tg = 1; tg < TG; ++tg) sum_vs = hadd_f16x2(sum_vs, hadd_f16x2(vs[tg][0], vs[tg][1]));
      const bool poisoned = __any_sync(0xffffffffu, any_nan_f16x2(sum_vs));

      if (!full || poisoned) {
        bool nan[TG][2];
#pragma unroll
        for (int tg = 0; tg < TG; ++tg)
#pragma unroll
          for (int hr = 0; hr < 2; ++hr)
            nan[tg][hr] = (st[kVs + (tg * 16 + kv4_perm(g8) + 8 * hr) * kScale] & 0x7fu) == 0x7fu;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int cc = 0; cc < 2; ++cc) {
            const int sees = row_keys(nt * 8 + 2 * t4 + cc) - key0;
            const int at = cur.block * R + nt * 8 + 2 * t4 + cc;
            // whether the row sees its tree's node at key `key` (past those that it sees all)
            auto node_seen = [&](int key) {
              const int m = key0 + key - (cur.req.keys - cur.req.queries);
              if (!TREE || m < 0 || key0 + key >= cur.req.keys || m >= 32 * a.words || at >= cur.req.q_len * a.group)
                return false;
              return (a.tree[static_cast<size_t>(cur.req.q0 + at / a.group) * a.words + m / 32] >> (m % 32) & 1u) != 0u;
            };
#pragma unroll
            for (int tg = 0; tg < TG; ++tg)
#pragma unroll
              for (int hr = 0; hr < 2; ++hr) {
                float& y = x[tg][nt][2 * hr + cc];
                if (nan[tg][hr]) y = __uint_as_float(0x7fffffffu);
                const int key = tg * 16 + kv4_perm(g8) + 8 * hr;
                if (!((have >> tg) & 1u) || (key >= sees && !node_seen(key))) y = -INFINITY;
              }
          }
#pragma unroll
        for (int tg = 0; tg < TG; ++tg) {
#pragma unroll
          for (int pr = 0; pr < 2; ++pr) {
            const float2 f = f16x2_to_f32x2(vs[tg][pr]);
            vs[tg][pr] = pack_f16x2(f.x == f.x ? f.x : 0.f, f.y == f.y ? f.y : 0.f);
          }
        }
      }

      // ---- softmax over the strip
      bool grow = false;
      float top[NT][2];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int cc = 0; cc < 2; ++cc) {
          top[nt][cc] = fmaxf(x[0][nt][cc], x[0][nt][2 + cc]);
#pragma unroll
          for (int tg = 1; tg < TG; ++tg) top[nt][cc] = max3f(top[nt][cc], x[tg][nt][cc], x[tg][nt][2 + cc]);
          grow |= top[nt][cc] > m[nt][cc] + kDecLazy;
        }
      if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int cc = 0; cc < 2; ++cc) {
            float v = top[nt][cc];
#pragma unroll
            for (int s = 4; s <= 16; s *= 2) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, s));
            v = fmaxf(v - kDecBelow, m[nt][cc]);
            const float alpha = ex2_mufu(m[nt][cc] - v);
            m[nt][cc] = v;
            l[nt][cc] *= alpha;
#pragma unroll
            for (int i = 0; i < MT; ++i) {
              o[i][nt][cc] *= alpha;
              o[i][nt][2 + cc] *= alpha;
            }
          }
      }
      uint32_t pb[TG][NT][2];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        const float2 below = f32x2(-m[nt][0], -m[nt][1]);
        float2 sum = f32x2(l[nt][0], l[nt][1]);
#pragma unroll
        for (int tg = 0; tg < TG; ++tg) {
#pragma unroll
          for (int hr = 0; hr < 2; ++hr) {
            const float2 y = add_f32x2(f32x2(x[tg][nt][2 * hr], x[tg][nt][2 * hr + 1]), below);
            const float2 p = f32x2(ex2_mufu(y.x), ex2_mufu(y.y));
            sum = add_f32x2(sum, p);
            pb[tg][nt][hr] = movmatrix_trans(pack_f16x2(p.x, p.y));
          }
        }
        l[nt][0] = sum.x;
        l[nt][1] = sum.y;
      }

      // ---- O^T += V^T P^T
#pragma unroll
      for (int tg = 0; tg < TG; ++tg) {
        uint32_t vw[4][VW];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const uint8_t* p = st + kV + (tg * 16 + kv4_perm(2 * t4 + (e & 1)) + 8 * (e >> 1)) * kCode;
          if constexpr (D == 128)
            *reinterpret_cast<uint2*>(vw[e]) = *reinterpret_cast<const uint2*>(p + g8 * 8);
          else
            vw[e][0] = *reinterpret_cast<const uint32_t*>(p + g8 * 4);
        }
#pragma unroll
        for (int w = 0; w < VW; ++w) {
          uint32_t even[2][4], odd[2][4];  // [token pair][dim pair]: dims 2i and 2i + 1
#pragma unroll
          for (int pr = 0; pr < 2; ++pr) {
            const uint32_t xa = vw[2 * pr][w], xb = vw[2 * pr + 1][w];
            unpack_e2m1x8((xa & 0x0f0f0f0fu) | ((xb << 4) & 0xf0f0f0f0u), even[pr]);
            unpack_e2m1x8(((xa >> 4) & 0x0f0f0f0fu) | (xb & 0xf0f0f0f0u), odd[pr]);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              even[pr][e] = mul_f16x2(even[pr][e], vs[tg][pr]);
              odd[pr][e] = mul_f16x2(odd[pr][e], vs[tg][pr]);
            }
          }
#pragma unroll
          for (int e = 0; e < 4; ++e)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
              mma_16816(o[4 * w + e][nt], even[0][e], odd[0][e], even[1][e], odd[1][e], pb[tg][nt][0],
                        pb[tg][nt][1]);
        }
      }
    }
    __syncwarp();
    issue(stage);
    stage = stage + 1 == kDecStages ? 0 : stage + 1;

    // ---- end of the unit, or of the CTA's share of it
    const bool unit_ends = cur.tile + 1 == cur.tiles;
    if (unit_ends || step + 1 == steps) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int cc = 0; cc < 2; ++cc) {
#pragma unroll
          for (int s = 4; s <= 16; s *= 2) l[nt][cc] += __shfl_xor_sync(0xffffffffu, l[nt][cc], s);
          if (g8 == 0) {
            s_m[warp][nt * 8 + 2 * t4 + cc] = m[nt][cc];
            s_l[warp][nt * 8 + 2 * t4 + cc] = l[nt][cc];
          }
        }
#pragma unroll
      for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
          area[((warp * MT + i) * NT + nt) * 32 + lane] =
              make_float4(o[i][nt][0], o[i][nt][1], o[i][nt][2], o[i][nt][3]);
      __syncthreads();  // (the one at the next unit's start keeps its sums out until all have read these)
      // Each warp adds up a quarter of the 16-dim tiles: the lanes' own places of all four warps.
      const bool complete = unit_ends && whole_start;
      const ReqShape req = cur.req;
      const int head = cur.head, row0 = cur.block * R, rows = req.q_len * a.group;
      const int slot = 2 * static_cast<int>(blockIdx.x) + (unit_no > 0 ? 1 : 0);
      constexpr int kMine = MT / kDecWarps;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        float f[kDecWarps][2], big[2], sum[2];
#pragma unroll
        for (int cc = 0; cc < 2; ++cc) {
          const int col = nt * 8 + 2 * t4 + cc;
          big[cc] = kDecNone;
          sum[cc] = 0.f;
#pragma unroll
          for (int w = 0; w < kDecWarps; ++w) big[cc] = fmaxf(big[cc], s_m[w][col]);
#pragma unroll
          for (int w = 0; w < kDecWarps; ++w) {
            f[w][cc] = ex2_mufu(s_m[w][col] - big[cc]);
            sum[cc] = fmaf(s_l[w][col], f[w][cc], sum[cc]);
          }
        }
        float y[kMine][4];
#pragma unroll
        for (int i = 0; i < kMine; ++i) {
#pragma unroll
          for (int e = 0; e < 4; ++e) y[i][e] = 0.f;
#pragma unroll
          for (int w = 0; w < kDecWarps; ++w) {
            const float4 x = area[((w * MT + warp * kMine + i) * NT + nt) * 32 + lane];
            y[i][0] = fmaf(x.x, f[w][0], y[i][0]);
            y[i][1] = fmaf(x.y, f[w][1], y[i][1]);
            y[i][2] = fmaf(x.z, f[w][0], y[i][2]);
            y[i][3] = fmaf(x.w, f[w][1], y[i][3]);
          }
        }
#pragma unroll
        for (int cc = 0; cc < 2; ++cc) {
          const int row = nt * 8 + 2 * t4 + cc;
          if (row0 + row >= rows) continue;
          const int dim = g8 * (D / 8) + warp * kMine * 2;  // the lane's 2 kMine dims
          if (complete) {
            const int qi = (row0 + row) / a.group, qg = row0 + row - qi * a.group;
            const size_t at = static_cast<size_t>(req.q0 + qi) * a.hq + head * a.group + qg;
            // nothing seen: O = 0 (a NaN sum stays NaN)
            const float inv = sum[cc] == 0.f ? 0.f : a.v_descale / sum[cc];
            uint32_t p[kMine];
#pragma unroll
            for (int i = 0; i < kMine; ++i) p[i] = pack_bf16x2(y[i][cc] * inv, y[i][2 + cc] * inv);
            if constexpr (kMine == 2)
              *reinterpret_cast<uint2*>(a.o + at * D + dim) = make_uint2(p[0], p[1]);
            else
              *reinterpret_cast<uint32_t*>(a.o + at * D + dim) = p[0];
            if (g8 == 0 && warp == 0)
              a.lse[at] = sum[cc] == 0.f ? -INFINITY : big[cc] * kLn2F + logf(sum[cc]);
          } else {
            float* dst = a.part_o + (static_cast<size_t>(slot) * R + row) * D + dim;
#pragma unroll
            for (int i = 0; i < kMine; ++i)
              *reinterpret_cast<float2*>(dst + 2 * i) = make_float2(y[i][cc], y[i][2 + cc]);
            if (g8 == 0 && warp == 0) a.part_ml[static_cast<size_t>(slot) * R + row] = make_float2(big[cc], sum[cc]);
          }
        }
      }
      if (whole_start && !unit_ends) {
        // the unit begins here and ends in a later CTA: x is its last tile on the line
        const long long x = first + step + (cur.tiles - 1 - cur.tile);
        merge = merge_desc(req, head, row0, min(R, rows - row0), slot,
                           share_of(total, n_cta, x) - static_cast<int>(blockIdx.x) + 1);
      }
      ++unit_no;
      fresh = true;
      whole_start = true;
    }
    if (step + 1 < steps) (void)cursor_next<D, R>(a, cur);
  }
  cp_async_wait<0>();
  if (threadIdx.x == 0 && !a.whole_tiles) a.desc[blockIdx.x] = merge;
}

// Merge of units that cross CTAs, launched while the attention kernel still runs.  The blocks (i, *)
// share the rows of the unit that begins in CTA i and ends in a later one, if there is one, or
// (`ctas` > 0, where few of all CTAs begin such a unit) of the i-th one that there is.  Of a unit
// in up to eight parts each warp takes rows of its own; of one in more parts a block takes a row
// and its warps share the parts.  Always summed in the same order.  Its time is latency (descriptor,
// then maxima and sums of the parts together): all loads of a row are in flight at once.
// It adds 3 us to a call for 64 requests, and 4 where the units of one are in 114 parts each.
constexpr int kMergeThreads = 256, kMergeWarps = kMergeThreads / 32;

template <int N>
__device__ __forceinline__ void load_floats(const float* src, float (&y)[N]) {
  if constexpr (N == 4)
    *reinterpret_cast<float4*>(y) = *reinterpret_cast<const float4*>(src);
  else
    *reinterpret_cast<float2*>(y) = *reinterpret_cast<const float2*>(src);
}

template <int D>
struct MergeShared {
  float m[kMergeWarps], l[kMergeWarps], o[kMergeWarps][D];
};

template <int D, int R>
__device__ __forceinline__ void kv4_merge_unit(const Kv4Args& a, const int4 u, MergeShared<D>& sh) {
  constexpr int kPer = D / 32;
  constexpr int kRows = R > 32 ? 4 : 1;  // rows that a warp takes at a time
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  const int first = u.x & 0xffff, parts = u.x >> 16, head = u.w & 0xffff, rows = u.w >> 16;
  // part k of row 0: the first CTA's, then the first of each later one
  auto slot = [&](int k) { return static_cast<size_t>(k == 0 ? first : (first & ~1) + 2 * k) * R; };
  auto store = [&](int row, float top, float sum, const float (&acc)[kPer]) {
    const int at_row = u.z + row, qi = at_row / a.group, qg = at_row - qi * a.group;
    const size_t to = static_cast<size_t>(u.y + qi) * a.hq + head * a.group + qg;
    const float inv = sum == 0.f ? 0.f : a.v_descale / sum;
    uint32_t p[kPer / 2];
#pragma unroll
    for (int e = 0; e < kPer / 2; ++e) p[e] = pack_bf16x2(acc[2 * e] * inv, acc[2 * e + 1] * inv);
    if constexpr (kPer == 4)
      *reinterpret_cast<uint2*>(a.o + to * D + lane * kPer) = make_uint2(p[0], p[1]);
    else
      *reinterpret_cast<uint32_t*>(a.o + to * D + lane * kPer) = p[0];
    if (lane == 0) a.lse[to] = sum == 0.f ? -INFINITY : top * kLn2F + logf(sum);
  };

  if (parts <= kMergeWarps) {
    constexpr int kAhead = kRows == 1 ? kMergeWarps : 2;  // parts whose sums are loaded together
    for (int row0 = (blockIdx.y * kMergeWarps + warp) * kRows; row0 < rows; row0 += gridDim.y * kMergeWarps * kRows) {
      const int n = min(kRows, rows - row0);
      // lane 8 r + k: row r, part k
      const int my_row = lane / 8, my_part = lane % 8;
      float2 ml = make_float2(kDecNone, 0.f);
      if (my_row < n && my_part < parts) ml = a.part_ml[slot(my_part) + row0 + my_row];
      float acc[kRows][kPer];
#pragma unroll
      for (int r = 0; r < kRows; ++r)
#pragma unroll
        for (int e = 0; e < kPer; ++e) acc[r][e] = 0.f;
      float top = ml.x;
#pragma unroll
      for (int k0 = 0; k0 < kMergeWarps; k0 += kAhead) {
        if (k0 >= parts) break;
        float y[kAhead][kRows][kPer];
#pragma unroll
        for (int k = 0; k < kAhead; ++k)
#pragma unroll
          for (int r = 0; r < kRows; ++r) {
#pragma unroll
            for (int e = 0; e < kPer; ++e) y[k][r][e] = 0.f;
            if (k0 + k < parts && r < n) load_floats(a.part_o + (slot(k0 + k) + row0 + r) * D + lane * kPer, y[k][r]);
          }
        if (k0 == 0) {
#pragma unroll
          for (int o = 1; o < 8; o *= 2) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
          ml.x = ex2_mufu(ml.x - top);
          ml.y *= ml.x;
#pragma unroll
          for (int o = 1; o < 8; o *= 2) ml.y += __shfl_xor_sync(0xffffffffu, ml.y, o);
        }
#pragma unroll
        for (int k = 0; k < kAhead; ++k)
#pragma unroll
          for (int r = 0; r < kRows; ++r) {
            const float f = __shfl_sync(0xffffffffu, ml.x, 8 * r + k0 + k);
#pragma unroll
            for (int e = 0; e < kPer; ++e) acc[r][e] = fmaf(y[k][r][e], f, acc[r][e]);
          }
      }
#pragma unroll
      for (int r = 0; r < kRows; ++r) {
        const float t = __shfl_sync(0xffffffffu, top, 8 * r), sum = __shfl_sync(0xffffffffu, ml.y, 8 * r);
        if (r < n) store(row0 + r, t, sum, acc[r]);
      }
    }
    return;
  }
  for (int row = blockIdx.y; row < rows; row += gridDim.y) {
    // the warp's parts warp, warp + 8, ...: 32 of them at a time, lane j part j
    float top = kDecNone, sum = 0.f, acc[kPer];
#pragma unroll
    for (int e = 0; e < kPer; ++e) acc[e] = 0.f;
    for (int k0 = warp; k0 < parts; k0 += 32 * kMergeWarps) {
      const int mine = k0 + lane * kMergeWarps;
      float2 ml = make_float2(kDecNone, 0.f);
      if (mine < parts) ml = a.part_ml[slot(mine) + row];
      float big = fmaxf(ml.x, top);
#pragma unroll
      for (int o = 1; o < 32; o *= 2) big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, o));
      const float f = ex2_mufu(ml.x - big), g = ex2_mufu(top - big);
      ml.y *= f;
#pragma unroll
      for (int o = 1; o < 32; o *= 2) ml.y += __shfl_xor_sync(0xffffffffu, ml.y, o);
      sum = fmaf(sum, g, ml.y);
      top = big;
#pragma unroll
      for (int e = 0; e < kPer; ++e) acc[e] *= g;
      const int here = min(32, (parts - k0 - 1) / kMergeWarps + 1);
      for (int j0 = 0; j0 < here; j0 += 16) {
        float y[16][kPer];
#pragma unroll
        for (int j = 0; j < 16; ++j) {
#pragma unroll
          for (int e = 0; e < kPer; ++e) y[j][e] = 0.f;
          if (j0 + j < here) load_floats(a.part_o + (slot(k0 + (j0 + j) * kMergeWarps) + row) * D + lane * kPer, y[j]);
        }
#pragma unroll
        for (int j = 0; j < 16; ++j) {
          const float fj = __shfl_sync(0xffffffffu, f, j0 + j);
#pragma unroll
          for (int e = 0; e < kPer; ++e) acc[e] = fmaf(y[j][e], fj, acc[e]);
        }
      }
    }
    if (lane == 0) sh.m[warp] = top;
    __syncthreads();
    const float own = top;
#pragma unroll
    for (int w = 0; w < kMergeWarps; ++w) top = fmaxf(top, sh.m[w]);
    const float f = ex2_mufu(own - top);
#pragma unroll
    for (int e = 0; e < kPer; ++e) sh.o[warp][lane * kPer + e] = acc[e] * f;
    if (lane == 0) sh.l[warp] = sum * f;
    __syncthreads();
    if (warp == 0) {
      sum = 0.f;
#pragma unroll
      for (int e = 0; e < kPer; ++e) acc[e] = 0.f;
#pragma unroll
      for (int w = 0; w < kMergeWarps; ++w) {
        sum += sh.l[w];
#pragma unroll
        for (int e = 0; e < kPer; ++e) acc[e] += sh.o[w][lane * kPer + e];
      }
      store(row, top, sum, acc);
    }
    __syncthreads();
  }
}

template <int D, int R>
__global__ void __launch_bounds__(kMergeThreads) kv4_merge_kernel(const Kv4Args a, int ctas) {
  __shared__ MergeShared<D> sh;
  grid_launch_dependents();
  grid_wait();
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  __shared__ int s_count[2][kMergeWarps], s_begins[2 * kMergeThreads];
  int units = 1;
  if (ctas > 0) {
    int before[2];
    unsigned begin[2];
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      const int i = x * kMergeThreads + threadIdx.x;
      begin[x] = __ballot_sync(0xffffffffu, i < ctas && a.desc[i].x >= 0);
      if (lane == 0) s_count[x][warp] = __popc(begin[x]);
    }
    __syncthreads();
    units = 0;
#pragma unroll
    for (int x = 0; x < 2; ++x)
#pragma unroll
      for (int w = 0; w < kMergeWarps; ++w) {
        if (w == warp) before[x] = units;
        units += s_count[x][w];
      }
#pragma unroll
    for (int x = 0; x < 2; ++x)
      if (begin[x] >> lane & 1u)
        s_begins[before[x] + __popc(begin[x] & ((1u << lane) - 1u))] = x * kMergeThreads + threadIdx.x;
    __syncthreads();
    units = (units - static_cast<int>(blockIdx.x) + static_cast<int>(gridDim.x) - 1) / static_cast<int>(gridDim.x);
  }
#pragma unroll 1
  for (int x = 0; x < units; ++x) {
    const int4 u = a.desc[ctas > 0 ? s_begins[blockIdx.x + x * gridDim.x] : blockIdx.x];
    if (u.x >= 0) kv4_merge_unit<D, R>(a, u, sh);
  }
}

}  // namespace exattn
