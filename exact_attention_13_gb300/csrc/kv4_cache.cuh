// kv4_cache.cuh -- the paged 4-bit key/value cache: layout, write, read back.
//
// Format.  A head vector is cut into groups of 16 values; a group holds one e4m3 scale and 16 e2m1
// codes (the magnitudes 0, 1/2, 1, 3/2, 2, 3, 4, 6), 4.5 bits a value:
//     s = e4m3(max |x| / 6),   code = e2m1(x / s),   value = code * s * descale
// both roundings to nearest even, saturating; descale is one power of two per tensor, so dividing
// by it is exact.  s = 0 (a group below half of e4m3's smallest step) stores zeros.
// A head vector that holds a NaN or an infinity gets NaN scales throughout: it reads back as NaN
// instead of as a large finite number.  code * s has at most six significant bits, so it is exact
// in bf16 and in f16.
// The quotients decide exactly as in real arithmetic: max |x| / 6 and x / s are correctly rounded
// fp32 quotients of numbers of at most 8 significant bits; on a rounding boundary of e4m3 or e2m1
// they are exact, and off it by a relative 2^-9 or more, far above fp32's rounding.
//
// Layout.  cache[page][head][K, V][block]; a block is page_size rows of d / 2 code bytes (value 2i
// in the low, 2i + 1 in the high half of byte i), then page_size rows of d / 16 scale bytes: the
// keys and the values of a page's head are one contiguous run of page_size * 9 d / 8 bytes.  Slot s
// is row s % page_size of page s / page_size.
//
// Both kernels give one thread a group: 32 bytes of bf16 on one side, 8 code bytes and a scale byte
// on the other, neighbouring lanes holding neighbouring groups.  They are bound by memory (or, for
// a decode step's few rows, by the launch).
#pragma once

#include <cuda_bf16.h>
#include <cstdint>

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

struct Kv4Rows {
  const __nv_bfloat16* k;  // append: [T, H, d] in (strides in elements)
  const __nv_bfloat16* v;
  __nv_bfloat16* k_out;    // read: [T, H, d] out, contiguous
  __nv_bfloat16* v_out;
  uint8_t* cache;
  const int* slots;        // [T]
  long long k_row, k_head, v_row, v_head;
  long long total;         // T * H * 2 * (d / 16) groups
  int t, heads, page, pages;
  float k_descale, v_descale;
};

// Group g of (tensor n, token, head): where its codes and its scale live; false when the slot lies
// outside the cache (such rows are skipped).
template <int D>
__device__ __forceinline__ bool kv4_place(const Kv4Rows& a, int n, int token, int head, int g,
                                          size_t& codes, size_t& scale) {
  const int slot = a.slots[token];
  if (slot < 0 || slot / a.page >= a.pages) return false;
  const int page = slot / a.page, row = slot - page * a.page;
  const size_t block = (static_cast<size_t>(page) * a.heads + head) * 2 + n;
  const size_t base = block * kv4_block_bytes(a.page, D);
  codes = base + row * (D / 2) + g * 8;
  scale = base + a.page * (D / 2) + row * (D / kKv4Group) + g;
  return true;
}

template <int D>
__global__ void __launch_bounds__(kKv4Threads) kv4_append_kernel(const Kv4Rows a) {
  constexpr int kGroups = D / kKv4Group;  // 8 or 4 neighbouring lanes hold one head vector
  const long long id = static_cast<long long>(blockIdx.x) * kKv4Threads + threadIdx.x;
  const bool live = id < a.total;
  const long long i = live ? id : a.total - 1;  // idle lanes repeat the last group, for the shuffles
  const int g = static_cast<int>(i % kGroups);
  const long long vec = i / kGroups;
  const int head = static_cast<int>(vec % a.heads);
  const long long row = vec / a.heads;
  const int n = row >= a.t ? 1 : 0;
  const int token = static_cast<int>(n ? row - a.t : row);

  const __nv_bfloat16* src = n ? a.v + token * a.v_row + head * a.v_head
                               : a.k + token * a.k_row + head * a.k_head;
  const uint4* p = reinterpret_cast<const uint4*>(src + g * kKv4Group);
  float x[2][8];
  unpack_bf16x8(__ldg(p), x[0]);
  unpack_bf16x8(__ldg(p + 1), x[1]);
  const float inv = 1.f / (n ? a.v_descale : a.k_descale);  // a power of two: exact
  float amax = 0.f;
  bool odd = false;
#pragma unroll
  for (int j = 0; j < 16; ++j) {
    float& f = x[j / 8][j % 8];
    odd |= !(fabsf(f) < INFINITY);
    f *= inv;
    amax = fmaxf(amax, fabsf(f));
  }
  const unsigned mask = __ballot_sync(0xffffffffu, odd);
  const unsigned mine = ((1u << kGroups) - 1u) << (threadIdx.x % 32 / kGroups * kGroups);
  uint32_t s8 = pack_e4m3x4(__fdiv_rn(amax, 6.f), 0.f, 0.f, 0.f) & 0xffu;
  uint32_t code[2] = {0u, 0u};
  if (mask & mine) {
    s8 = 0x7fu;  // NaN
  } else if (s8 != 0u) {
    const float s = f16x2_to_f32x2(e4m3x2_to_f16x2(static_cast<uint16_t>(s8))).x;
#pragma unroll
    for (int j = 0; j < 16; ++j) x[j / 8][j % 8] = __fdiv_rn(x[j / 8][j % 8], s);
    code[0] = pack_e2m1x8(x[0]);
    code[1] = pack_e2m1x8(x[1]);
  }
  size_t codes, scale;
  if (live && kv4_place<D>(a, n, token, head, g, codes, scale)) {
    *reinterpret_cast<uint2*>(a.cache + codes) = make_uint2(code[0], code[1]);
    a.cache[scale] = static_cast<uint8_t>(s8);
  }
}

// Rows of invalid slots read as zeros.
template <int D>
__global__ void __launch_bounds__(kKv4Threads) kv4_read_kernel(const Kv4Rows a) {
  constexpr int kGroups = D / kKv4Group;
  const long long i = static_cast<long long>(blockIdx.x) * kKv4Threads + threadIdx.x;
  if (i >= a.total) return;
  const int g = static_cast<int>(i % kGroups);
  const long long vec = i / kGroups;
  const int head = static_cast<int>(vec % a.heads);
  const long long row = vec / a.heads;
  const int n = row >= a.t ? 1 : 0;
  const int token = static_cast<int>(n ? row - a.t : row);
  uint4 out[2] = {make_uint4(0u, 0u, 0u, 0u), make_uint4(0u, 0u, 0u, 0u)};
  size_t codes, scale;
  if (kv4_place<D>(a, n, token, head, g, codes, scale)) {
    const uint2 c = *reinterpret_cast<const uint2*>(a.cache + codes);
    const float s = f16x2_to_f32x2(e4m3x2_to_f16x2(a.cache[scale])).x *
                    (n ? a.v_descale : a.k_descale);
    const uint32_t w[2] = {c.x, c.y};
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      uint32_t h[4];
      unpack_e2m1x8(w[q], h);
      float f[8];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float2 two = f16x2_to_f32x2(h[j]);
        f[2 * j] = two.x * s;
        f[2 * j + 1] = two.y * s;
      }
      out[q] = pack_bf16x8(f);
    }
  }
  __nv_bfloat16* dst = (n ? a.v_out : a.k_out) +
                       (static_cast<size_t>(token) * a.heads + head) * D + g * kKv4Group;
  reinterpret_cast<uint4*>(dst)[0] = out[0];
  reinterpret_cast<uint4*>(dst)[1] = out[1];
}

}  // namespace exattn
