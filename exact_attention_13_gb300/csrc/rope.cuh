// rope.cuh -- rotary positions for the attention operands.
//
// Pair i of a head vector at position p is turned by the angle p f_i:
//     y_a = m (a cos - b sin),   y_b = m (b cos + a sin)
// with (a, b) = (x_i, x_{i + r/2}) (halves) or (x_{2i}, x_{2i+1}) (interleaved), r rotated values
// per head; the rest of the head passes through.  The map is m times a rotation, so its gradient
// is the same map with -p f_i (the `inverse` flag).
//
// Angles.  p f_i in fp32 is off by up to 2^-24 p f_i radians: at position 2^17 already 2^-7.  The
// step f_i is therefore held as a 64-bit fixed-point fraction of a turn (unit 2^-64 turn), and
// p * step in wrapping 64-bit integer arithmetic IS the fractional part of the angle in turns:
// the whole turns drop out of the product by themselves.  The step's rounding (2^-65 turn in a table made
// with enough digits; one made in doubles is off by up to 2^-55) times p < 2^31 leaves at most 2^-34
// turn; the top 32 bits, rounded to fp32, go to sincospif (2^-25 of
// half a turn).  Arithmetic is fp32, one rounding to bf16 at the end.
//
// One thread owns one row (batch, position) and one 16-value chunk of the head -- eight pairs, two
// 16-byte loads and stores per head -- and walks over a range of heads, so its eight angles are
// computed once.  The D / 16 chunks of a row sit in neighbouring lanes: a warp moves whole
// 128-byte lines.  Bound by memory: 537 MB (B 2, 32 + 32 heads, N 8192, d 128) take 78.8 us, 6.8 TB/s.
//
// Several axes (AXES): the tokens of images and video have a position on each of up to four axes (time,
// height, width), and each pair turns by its own axis's: p is p_{axis(i)}.  A row's positions are loaded once
// a thread, the eight pairs' axes as one word, and each pair selects its position: 16 % more ALU instructions than
// with one axis (51 % of their issue slots), 80.1 us instead of 78.8 for the 537 MB above.
#pragma once

#include <cuda_bf16.h>
#include <cstdint>

#include "sm103_ptx.cuh"

namespace exattn {

constexpr int kRopeThreads = 128;

// The kernels of a serving step follow each other at once: each is launched while the one before it
// still runs (as soon as all of that one's blocks have started), and waits for its end and
// its writes before it touches memory.  (Such a kernel's inputs may be written during its lifetime, so
// the loads are ordinary ones, not those of the non-coherent path.)
__device__ __forceinline__ void grid_launch_dependents() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}
__device__ __forceinline__ void grid_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

struct RopeTensor {
  const __nv_bfloat16* x;
  __nv_bfloat16* y;
  long long xb, xh, xn;  // strides in elements: batch, head, row
  long long yb, yh, yn;
  int heads;             // 0: no such tensor
};

struct RopeArgs {
  RopeTensor t[2];
  const int* positions;       // [B, N] (pos_batch = stride of B, 0 when shared)
  const long long* turns;     // [r / 2], units of 2^-64 turn
  long long pos_batch;
  long long rows;             // B * N
  int n;
  int d, r;
  float mscale;
  int heads_per_thread;
  const uint8_t* axes;        // [r / 2] axis of each pair; positions of axis x lie x * pos_axis on
  long long pos_axis;
  int n_axes;                 // 1 .. kRopeAxes
};
constexpr int kRopeAxes = 4;

__device__ __forceinline__ void unpack_bf16x8(const uint4& raw, float (&f)[8]) {
  const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __uint_as_float(w[i] << 16);
    f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
}

__device__ __forceinline__ uint4 pack_bf16x8(const float (&f)[8]) {
  return make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                    pack_bf16x2(f[6], f[7]));
}

template <bool INTERLEAVED, bool INVERSE, bool AXES>
__global__ void __launch_bounds__(kRopeThreads) rope_kernel(const RopeArgs a) {
  grid_launch_dependents();
  grid_wait();
  const int chunks = a.d / 16;
  const long long id = static_cast<long long>(blockIdx.x) * kRopeThreads + threadIdx.x;
  const long long row = id / chunks;
  if (row >= a.rows) return;
  const int chunk = static_cast<int>(id - row * chunks);
  const int batch = static_cast<int>(row / a.n);
  const int n = static_cast<int>(row - static_cast<long long>(batch) * a.n);
  const bool rotate = chunk < a.r / 16;
  // element offsets of the thread's two 8-value pieces
  const int e0 = INTERLEAVED || !rotate ? chunk * 16 : chunk * 8;
  const int e1 = INTERLEAVED || !rotate ? e0 + 8 : a.r / 2 + e0;

  float cs[8], sn[8];
  if (rotate) {
    const int* at = a.positions + batch * a.pos_batch + n;
    int pos[AXES ? kRopeAxes : 1];
    uint2 axes = make_uint2(0u, 0u);
    pos[0] = at[0];
    if constexpr (AXES) {
#pragma unroll
      for (int x = 1; x < kRopeAxes; ++x) pos[x] = x < a.n_axes ? at[x * a.pos_axis] : pos[0];
      axes = *reinterpret_cast<const uint2*>(a.axes + chunk * 8);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      int mine = pos[0];
      if constexpr (AXES) {  // (an axis that there is not: the first one)
        const uint32_t axis = ((i < 4 ? axes.x : axes.y) >> (i % 4 * 8)) & 0xffu;
#pragma unroll
        for (int x = 1; x < kRopeAxes; ++x) mine = axis == static_cast<uint32_t>(x) ? pos[x] : mine;
      }
      const unsigned long long p = static_cast<unsigned long long>(static_cast<long long>(mine));
      const unsigned long long turn = p * static_cast<unsigned long long>(a.turns[chunk * 8 + i]);
      // fraction of a turn in [-1/2, 1/2), as half turns
      const float half_turns = __int2float_rn(static_cast<int>(turn >> 32)) * 0x1p-31f;
      sincospif(half_turns, &sn[i], &cs[i]);
      cs[i] *= a.mscale;
      sn[i] *= INVERSE ? -a.mscale : a.mscale;
    }
  }

  const int total = a.t[0].heads + a.t[1].heads;
  const int h0 = blockIdx.y * a.heads_per_thread;
  const int h1 = min(total, h0 + a.heads_per_thread);
  constexpr int kUnroll = 4;  // heads whose loads are in flight together
  for (int h = h0; h < h1; h += kUnroll) {
    uint4 in0[kUnroll], in1[kUnroll];
    __nv_bfloat16* out[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      if (h + u < h1) {
        const bool second = h + u >= a.t[0].heads;
        const RopeTensor& t = a.t[second ? 1 : 0];
        const int hh = h + u - (second ? a.t[0].heads : 0);
        const __nv_bfloat16* src = t.x + batch * t.xb + hh * t.xh + n * t.xn;
        out[u] = t.y + batch * t.yb + hh * t.yh + n * t.yn;
        in0[u] = *reinterpret_cast<const uint4*>(src + e0);
        in1[u] = *reinterpret_cast<const uint4*>(src + e1);
      }
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      if (h + u < h1) {
        if (rotate) {
          float x0[8], x1[8];
          unpack_bf16x8(in0[u], x0);
          unpack_bf16x8(in1[u], x1);
          if constexpr (INTERLEAVED) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const float p0 = x0[2 * i], p1 = x0[2 * i + 1];
              x0[2 * i] = fmaf(p0, cs[i], -p1 * sn[i]);
              x0[2 * i + 1] = fmaf(p1, cs[i], p0 * sn[i]);
              const float q0 = x1[2 * i], q1 = x1[2 * i + 1];
              x1[2 * i] = fmaf(q0, cs[4 + i], -q1 * sn[4 + i]);
              x1[2 * i + 1] = fmaf(q1, cs[4 + i], q0 * sn[4 + i]);
            }
          } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const float p0 = x0[i], p1 = x1[i];
              x0[i] = fmaf(p0, cs[i], -p1 * sn[i]);
              x1[i] = fmaf(p1, cs[i], p0 * sn[i]);
            }
          }
          in0[u] = pack_bf16x8(x0);
          in1[u] = pack_bf16x8(x1);
        }
        *reinterpret_cast<uint4*>(out[u] + e0) = in0[u];
        *reinterpret_cast<uint4*>(out[u] + e1) = in1[u];
      }
    }
  }
}

}  // namespace exattn
