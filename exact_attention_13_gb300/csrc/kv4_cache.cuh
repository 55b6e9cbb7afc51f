// kv4_cache.cuh -- the paged 4-bit key/value cache: layout, write, read back, move of rows.
//
// Format.  A head vector is cut into groups of 16 values; a group holds one e4m3 scale and 16 e2m1
// codes (the magnitudes 0, 1/2, 1, 3/2, 2, 3, 4, 6), 4.5 bits a value:
//     s = e4m3(max |x| / 6),   code = e2m1(x / s),   value = code * s * descale
// both roundings to nearest even, saturating; descale is one power of two per tensor, so dividing
// by it is exact.  s = 0 (a group below half of e4m3's smallest step) stores zeros.
// A head vector that holds a NaN or an infinity gets NaN scales throughout: it reads back as NaN
// instead of as a large finite number.  code * s has at most six significant bits, so it is exact
// in bf16 and in f16.
// The roundings decide exactly as in real arithmetic, without divisions.  A midpoint of e4m3 times 6
// has at most 7 significant bits and max |x| has 8, so max |x| / 6 lies on a midpoint or a relative
// 2^-8 off it.  The product with 1/6 is off by 2^-23; rounding it to f16 first (2^-12) brings the
// former onto the midpoint, which f16 holds, and leaves the latter on its side.  Likewise x / s lies
// on a midpoint of e2m1 (a multiple of 2^-2) or a relative 2^-8 off it; the product with the
// reciprocal of s (off by 2^-22) is rounded to the grid of 2^-14, which moves it by 2^-15, less than a
// tenth of that distance at the smallest midpoint, 1/4.  (17 divisions a group took most of the
// instructions.)
//
// Layout.  cache[page][head][K, V][block]; a block is page_size rows of d / 2 code bytes (value 2i
// in the low, 2i + 1 in the high half of byte i), then page_size rows of d / 16 scale bytes: the
// keys and the values of a page's head are one contiguous run of page_size * 9 d / 8 bytes.  Slot s
// is row s % page_size of page s / page_size.
//
// A thread of the append kernel takes the same group of the keys and of the values, one of the read
// kernel half of it: 8 values are 16 bytes of bf16, so the read kernel's stores are whole lines.
// (Groups in both: 11.2 us to read 8191 tokens of 8 heads of 128 from consecutive slots instead of
// 10.0; halves in both: 11.3 us to append them instead of the 9 of groups, whose code stores are
// twice as wide.)  A decode step's few rows are bound by the launch.  Those 8191 tokens (43 MB each way, 6.4 us)
// take 8.1 us to append and 9.9 to read in whole pages, bound by the chain slot, address, codes, store
// of one piece a thread; 12.6 and 12.3 at scattered slots, whose rows are short pieces of lines.
#pragma once

#include <cuda_bf16.h>
#include <cstdint>
#include <type_traits>

#include "rope.cuh"
#include "sm103_ptx.cuh"

namespace exattn {

constexpr int kKv4Group = 16;
constexpr int kKv4Threads = 128;

// Bytes of one (page, head, K or V) block.
__host__ __device__ constexpr int kv4_block_bytes(int page, int d) { return page * (d / 2 + d / kKv4Group); }

// Eight fp32 values to e2m1 (nearest even, saturating at 6), value i in bits 4i .. 4i+3.
__device__ __forceinline__ uint32_t pack_e2m1x8(const float* f) {
  uint32_t r;
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n\t"
      "mov.b32 %0, {b0, b1, b2, b3};\n\t}"
      : "=r"(r)
      : "f"(f[0]), "f"(f[1]), "f"(f[2]), "f"(f[3]), "f"(f[4]), "f"(f[5]), "f"(f[6]), "f"(f[7]));
  return r;
}

// The eight e2m1 codes of a word as f16 pairs: h[i] = values 2i (low half) and 2i + 1.
__device__ __forceinline__ void unpack_e2m1x8(uint32_t w, uint32_t (&h)[4]) {
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
      "mov.b32 {b0, b1, b2, b3}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, b0;\n\t"
      "cvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, b2;\n\t"
      "cvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
      : "r"(w));
}

// The f16 in the low half as e4m3 (nearest even, saturating).
__device__ __forceinline__ uint32_t e4m3_from_f16(uint32_t h) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(r) : "r"(h));
  return r & 0xffu;
}
// 1 / x, within 2^-23 of it.
__device__ __forceinline__ float rcp_approx(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

struct Kv4Rows {
  const __nv_bfloat16* in[2];   // append: keys and values [T, H, d] (strides in elements)
  __nv_bfloat16* out[2];        // read: [T, H, d], contiguous
  uint8_t* cache;
  const int* slots;             // [T]
  long long row[2], head[2];
  float descale[2];
  int pieces;                   // threads of this launch, T * H * (d / 16 or d / 8), below 2^31
  int heads, page_shift, pages;
};

// A thread's piece of kSize values: (token, head, piece of the head).
template <int D, int kSize>
struct Kv4Index {
  static constexpr int kPieces = D / kSize;
  int token, head, p;
  __device__ __forceinline__ Kv4Index(const Kv4Rows& a, int i) {
    const int vec = i / kPieces;
    p = i % kPieces;
    token = vec / a.heads;
    head = vec - token * a.heads;
  }
};

// Where its codes in the K block lie: the scale is `scale` bytes on, the V block `block` bytes on.
// at < 0: the slot lies outside the cache.
template <int D, int kSize>
struct Kv4Place {
  long long at;
  int scale, block;
  __device__ __forceinline__ Kv4Place(const Kv4Rows& a, const Kv4Index<D, kSize>& x, int slot) {
    const int page = slot >> a.page_shift, rows = 1 << a.page_shift, row = slot & (rows - 1);
    const int code = x.p * (kSize / 2);
    block = kv4_block_bytes(rows, D);
    scale = rows * (D / 2) + row * (D / kKv4Group - D / 2) + x.p * kSize / kKv4Group - code;
    at = slot < 0 || page >= a.pages
             ? -1
             : (static_cast<long long>(page) * a.heads + x.head) * 2 * block + row * (D / 2) + code;
  }
};

template <int D>
__global__ void __launch_bounds__(kKv4Threads) kv4_append_kernel(const Kv4Rows a) {
  grid_launch_dependents();
  grid_wait();
  using Index = Kv4Index<D, kKv4Group>;
  constexpr int kPieces = Index::kPieces;  // 8 or 4 neighbouring lanes hold one head vector
  const int id = blockIdx.x * kKv4Threads + threadIdx.x;
  const bool live = id < a.pieces;
  const Index ix(a, live ? id : a.pieces - 1);  // idle lanes repeat the last piece, for the votes
  const int slot = *(a.slots + ix.token);
  uint4 raw[2][2];
#pragma unroll
  for (int n = 0; n < 2; ++n) {
    const uint4* src = reinterpret_cast<const uint4*>(a.in[n] + ix.token * a.row[n] + ix.head * a.head[n]) + 2 * ix.p;
    raw[n][0] = *src;
    raw[n][1] = *(src + 1);
  }
  const Kv4Place<D, kKv4Group> place(a, ix, slot);
  const unsigned mine = ((1u << kPieces) - 1u) << (threadIdx.x % 32 / kPieces * kPieces);
#pragma unroll
  for (int n = 0; n < 2; ++n) {
    float x[16];
    unpack_bf16x8(raw[n][0], reinterpret_cast<float(&)[8]>(x[0]));
    unpack_bf16x8(raw[n][1], reinterpret_cast<float(&)[8]>(x[8]));
    // 0 x is 0 but for infinities and NaN
    float amax = 0.f;
    float2 odd = f32x2(0.f, 0.f);
#pragma unroll
    for (int j = 0; j < 16; j += 2) {
      amax = max3f(amax, fabsf(x[j]), fabsf(x[j + 1]));
      odd = fma_f32x2(f32x2(x[j], x[j + 1]), f32x2(0.f, 0.f), odd);
    }
    const unsigned bad = __ballot_sync(0xffffffffu, !(odd.x + odd.y == 0.f));
    const float inv_descale = 1.f / a.descale[n];
    // inv_descale is a power of two: the product with it is exact
    uint32_t s8 = e4m3_from_f16(pack_f16x2(amax * inv_descale * (1.f / 6.f), 0.f));
    uint32_t code[2] = {0u, 0u};
    if (bad & mine) {
      s8 = 0x7fu;  // NaN
    } else if (s8 != 0u) {
      const float s = f16x2_to_f32x2(e4m3x2_to_f16x2(static_cast<uint16_t>(s8))).x;
      const float inv = rcp_approx(s) * inv_descale;
      // 768 = 1.5 * 2^9: adding it rounds to multiples of 2^-14; the sign of zeros is put back
      const float2 inv2 = f32x2(inv, inv), up = f32x2(768.f, 768.f), down = f32x2(-768.f, -768.f);
#pragma unroll
      for (int j = 0; j < 16; j += 2) {
        const float2 t = add_f32x2(fma_f32x2(f32x2(x[j], x[j + 1]), inv2, up), down);
        x[j] = copysignf(t.x, x[j]);
        x[j + 1] = copysignf(t.y, x[j + 1]);
      }
      code[0] = pack_e2m1x8(x);
      code[1] = pack_e2m1x8(x + 8);
    }
    if (live && place.at >= 0) {
      uint8_t* dst = a.cache + place.at + n * place.block;
      *reinterpret_cast<uint2*>(dst) = make_uint2(code[0], code[1]);
      dst[place.scale] = static_cast<uint8_t>(s8);
    }
  }
}

// Rows of invalid slots read as zeros.
template <int D>
__global__ void __launch_bounds__(kKv4Threads) kv4_read_kernel(const Kv4Rows a) {
  grid_launch_dependents();
  grid_wait();
  const int id = blockIdx.x * kKv4Threads + threadIdx.x;
  if (id >= a.pieces) return;
  const Kv4Index<D, 8> ix(a, id);
  const Kv4Place<D, 8> place(a, ix, *(a.slots + ix.token));
  uint32_t codes[2] = {0u, 0u};
  uint8_t s8[2] = {0, 0};
  if (place.at >= 0) {
#pragma unroll
    for (int n = 0; n < 2; ++n) {
      const uint8_t* src = a.cache + place.at + n * place.block;
      codes[n] = *reinterpret_cast<const uint32_t*>(src);
      s8[n] = src[place.scale];
    }
  }
#pragma unroll
  for (int n = 0; n < 2; ++n) {
    const float s = f16x2_to_f32x2(e4m3x2_to_f16x2(s8[n])).x * a.descale[n];
    uint32_t h[4];
    unpack_e2m1x8(codes[n], h);
    float f[8];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float2 two = f16x2_to_f32x2(h[j]);
      f[2 * j] = two.x * s;
      f[2 * j + 1] = two.y * s;
    }
    reinterpret_cast<uint4*>(a.out[n])[id] = pack_bf16x8(f);
  }
}

// Rows of one cache, or of the caches of all layers, to other slots: of request r, row sources[i] to
// slots[i] for its first counts[r] rows i, in their order.  A row is D / 16 bytes of scales and eight times as
// much of codes: nine pieces of that size, of which a thread takes one, of the keys or the values of one head,
// through all of the request's rows.  Eight rows are read before they are written; in a path of accepted
// nodes, whose sources rise and lie at or behind their destinations, no source is then written before it is
// read.  Bound by latency (count, slots, row: 2.2 us for 8 requests and 4 layers), for large steps by short pieces
// of lines: 64 requests, 64 layers, 20 MB of rows take 15.3 us; their 64 + 8 bytes at random places are 96 of
// 32-byte sectors to read, 26.9 MB, and as much again to write.  47.5 MB are read from DRAM (3.3 TB/s); the counters do
// not show what the others are (fills of partly written sectors, perhaps, and a DRAM granule of two).
constexpr int kMoveLayers = 256;  // caches of one launch (their addresses are the kernel's arguments)
constexpr int kMoveAhead = 8;

struct Kv4MoveArgs {
  uint8_t* cache[kMoveLayers];
  const int* sources;   // [T]
  const int* slots;     // [T]
  const int* offsets;   // [B + 1]
  const int* counts;    // [B]
  int t, b, heads, page_shift, pages;
};

template <int D>
__global__ void __launch_bounds__(kKv4Threads) kv4_move_kernel(const __grid_constant__ Kv4MoveArgs a) {
  using Piece = typename std::conditional<D == 128, uint2, uint32_t>::type;
  constexpr int kPieces = 9;
  static_assert(sizeof(Piece) == D / kKv4Group, "a row of scales is one piece");
  grid_launch_dependents();
  grid_wait();
  unsigned id = blockIdx.x * kKv4Threads + threadIdx.x;
  const unsigned piece = id % kPieces;
  id /= kPieces;
  const unsigned r = id / (2u * a.heads), vec = id - r * (2u * a.heads);  // 2 head + (0 keys, 1 values)
  if (r >= static_cast<unsigned>(a.b)) return;
  const int first = min(max(a.offsets[r], 0), a.t);
  const int n = min(a.counts[r], min(max(a.offsets[r + 1], first), a.t) - first);
  const int rows = 1 << a.page_shift, block = kv4_block_bytes(rows, D);
  uint8_t* const base = a.cache[blockIdx.y] + static_cast<size_t>(vec) * block +
                        (piece < 8 ? piece * sizeof(Piece) : static_cast<unsigned>(rows) * (D / 2));
  const unsigned step = piece < 8 ? D / 2 : D / kKv4Group;
  const size_t page_bytes = static_cast<size_t>(block) * 2u * a.heads;
  auto place = [&](int slot) {
    return reinterpret_cast<Piece*>(base + static_cast<size_t>(slot >> a.page_shift) * page_bytes +
                                    static_cast<unsigned>(slot & (rows - 1)) * step);
  };
  auto there = [&](int slot) { return slot >= 0 && (slot >> a.page_shift) < a.pages; };
  for (int i0 = 0; i0 < n; i0 += kMoveAhead) {
    int from[kMoveAhead], to[kMoveAhead];
    Piece x[kMoveAhead];
#pragma unroll
    for (int i = 0; i < kMoveAhead; ++i) {
      const bool live = i0 + i < n;
      from[i] = live ? a.sources[first + i0 + i] : -1;
      to[i] = live ? a.slots[first + i0 + i] : -1;
    }
#pragma unroll
    for (int i = 0; i < kMoveAhead; ++i) {
      if (from[i] == to[i] || !there(from[i]) || !there(to[i])) to[i] = -1;
      if (to[i] >= 0) x[i] = *place(from[i]);
    }
#pragma unroll
    for (int i = 0; i < kMoveAhead; ++i)
      if (to[i] >= 0) *place(to[i]) = x[i];
  }
}

}  // namespace exattn
