// kv_api.cu -- host side of the operators around attention: rotary positions, page planning, the
// 4-bit key/value cache and attention over it.  Argument checks and launches of the C ABI declared
// in include/exact_attention.h; no call allocates, synchronises or throws.
#include <cuda_runtime.h>

#include <atomic>
#include <cmath>
#include <cstdint>
#include <initializer_list>

#include "../../include/exact_attention.h"
#include "kv4_cache.cuh"
#include "kv4_launch.cuh"
#include "kv_host.cuh"
#include "page_plan.cuh"
#include "rope.cuh"

namespace exattn {

namespace {

// ---------------------------------------------------------------------------------- rope
int rope_tensor(RopeTensor& t, const void* x, const long long* xs, void* y, const long long* ys,
                int heads) {
  t = RopeTensor{};
  if (heads == 0) return FA_OK;
  if (heads < 0 || !x || !y || !xs || !ys) return FA_ERR_INVALID_ARG;
  for (int i = 0; i < 3; ++i) {
    if (xs[i] < 0 || ys[i] < 0) return FA_ERR_INVALID_ARG;
    if (xs[i] % 8 || ys[i] % 8) return FA_ERR_MISALIGNED;
  }
  if (!aligned(x, 16) || !aligned(y, 16)) return FA_ERR_MISALIGNED;
  t.x = static_cast<const __nv_bfloat16*>(x);
  t.y = static_cast<__nv_bfloat16*>(y);
  t.xb = xs[0];
  t.xh = xs[1];
  t.xn = xs[2];
  t.yb = ys[0];
  t.yh = ys[1];
  t.yn = ys[2];
  t.heads = heads;
  return FA_OK;
}

// fa_rope, and (a.axes given) fa_rope_axes.
int launch_rope(RopeArgs& a, const void* q, const long long* q_strides, void* q_out, const long long* q_out_strides,
                int Hq, const void* k, const long long* k_strides, void* k_out, const long long* k_out_strides,
                int Hk, int B, int N, int d, const int* positions, long long positions_batch_stride,
                const long long* turns, int rotary_dim, int flags, float mscale, void* stream) {
  if (!positions || !turns || B < 1 || N < 1 || Hq < 1 || Hk < 0 || positions_batch_stride < 0)
    return FA_ERR_INVALID_ARG;
  if (flags & ~(FA_ROPE_INTERLEAVED | FA_ROPE_INVERSE)) return FA_ERR_INVALID_ARG;
  if (!std::isfinite(mscale)) return FA_ERR_INVALID_ARG;
  if (d != 64 && d != 128) return FA_ERR_UNSUPPORTED;
  if (rotary_dim < 16 || rotary_dim > d || rotary_dim % 16) return FA_ERR_UNSUPPORTED;
  if (!aligned(positions, 4) || !aligned(turns, 8)) return FA_ERR_MISALIGNED;
  if (int rc = rope_tensor(a.t[0], q, q_strides, q_out, q_out_strides, Hq)) return rc;
  if (int rc = rope_tensor(a.t[1], k, k_strides, k_out, k_out_strides, Hk)) return rc;
  a.positions = positions;
  a.turns = turns;
  a.pos_batch = positions_batch_stride;
  a.rows = static_cast<long long>(B) * N;
  a.n = N;
  a.d = d;
  a.r = rotary_dim;
  a.mscale = mscale;
  const long long blocks = (a.rows * (d / 16) + kRopeThreads - 1) / kRopeThreads;
  if (blocks > 0x7fffffffll || static_cast<long long>(Hq) + Hk > 65535) return FA_ERR_UNSUPPORTED;
  // Heads per thread: four, whose loads are in flight together.  (B2 H32+32 N8192 d128 takes 78.7 us
  // with 4, 79.9 with 8, 81.1 with 16 and 89.5 with all 64: the angles that more heads would share
  // cost less than the longer blocks' last wave.)  Fewer where that leaves less than eight blocks a
  // SM, as in a decode step.
  const int heads = Hq + Hk;
  a.heads_per_thread = 4;
  while (a.heads_per_thread > 1 &&
         blocks * ((heads + a.heads_per_thread - 1) / a.heads_per_thread) < 8 * kSms)
    a.heads_per_thread /= 2;
  const dim3 grid(static_cast<unsigned>(blocks),
                  static_cast<unsigned>((heads + a.heads_per_thread - 1) / a.heads_per_thread));
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const bool il = flags & FA_ROPE_INTERLEAVED, inv = flags & FA_ROPE_INVERSE;
  auto kern = a.axes ? il ? inv ? rope_kernel<true, true, true> : rope_kernel<true, false, true>
                          : inv ? rope_kernel<false, true, true> : rope_kernel<false, false, true>
                     : il ? inv ? rope_kernel<true, true, false> : rope_kernel<true, false, false>
                          : inv ? rope_kernel<false, true, false> : rope_kernel<false, false, false>;
  return launch_early(kern, grid, kRopeThreads, 0, s, a);
}

// ---------------------------------------------------------------------------------- cache
// Append or read T tokens, in launches of fewer than 2^31 pieces (32-bit indices).
int launch_rows(Kv4Rows a, int T, int heads, int d, int piece, void (*k64)(Kv4Rows), void (*k128)(Kv4Rows),
                cudaStream_t s) {
  const int per_token = heads * (d / piece);
  const int most = ((1 << 30) / per_token);
  for (int t = 0; t < T; t += most) {
    const int n = T - t < most ? T - t : most;
    a.pieces = n * per_token;
    const unsigned grid = static_cast<unsigned>((a.pieces + kKv4Threads - 1) / kKv4Threads);
    if (int rc = launch_early(d == 64 ? k64 : k128, grid, kKv4Threads, 0, s, a)) return rc;
    a.slots += n;
    for (int i = 0; i < 2; ++i) {
      if (a.in[i]) a.in[i] += n * a.row[i];
      if (a.out[i]) a.out[i] += static_cast<long long>(n) * heads * d;
    }
    if (T - t <= most) break;  // (t + most may pass 2^31)
  }
  return FA_OK;
}

// ---------------------------------------------------------------------------------- attention
template <int D>
int launch_kv4(Kv4Args& a, int nt, void* workspace, cudaStream_t s) {
  return nt == 0   ? launch_chunk<D>(a, workspace, s)
         : nt == 1 ? launch_decode<D, 1>(a, workspace, s)
         : nt == 2 ? launch_decode<D, 2>(a, workspace, s)
                   : launch_decode<D, 4>(a, workspace, s);
}

}  // namespace
}  // namespace exattn

using namespace exattn;

extern "C" {

int fa_rope(const void* q, const long long* q_strides, void* q_out, const long long* q_out_strides,
            int Hq, const void* k, const long long* k_strides, void* k_out,
            const long long* k_out_strides, int Hk, int B, int N, int d, const int* positions,
            long long positions_batch_stride, const long long* turns, int rotary_dim, int flags,
            float mscale, void* stream) {
  RopeArgs a{};
  return launch_rope(a, q, q_strides, q_out, q_out_strides, Hq, k, k_strides, k_out, k_out_strides, Hk, B, N, d,
                     positions, positions_batch_stride, turns, rotary_dim, flags, mscale, stream);
}

int fa_rope_axes(const void* q, const long long* q_strides, void* q_out, const long long* q_out_strides,
                 int Hq, const void* k, const long long* k_strides, void* k_out,
                 const long long* k_out_strides, int Hk, int B, int N, int d, const int* positions,
                 int num_axes, long long positions_axis_stride, long long positions_batch_stride,
                 const unsigned char* axes, const long long* turns, int rotary_dim, int flags, float mscale,
                 void* stream) {
  if (!axes || num_axes < 1 || positions_axis_stride < 0) return FA_ERR_INVALID_ARG;
  if (num_axes > kRopeAxes) return FA_ERR_UNSUPPORTED;
  if (!aligned(axes, 8)) return FA_ERR_MISALIGNED;
  RopeArgs a{};
  a.axes = axes;
  a.n_axes = num_axes;
  a.pos_axis = positions_axis_stride;
  return launch_rope(a, q, q_strides, q_out, q_out_strides, Hq, k, k_strides, k_out, k_out_strides, Hk, B, N, d,
                     positions, positions_batch_stride, turns, rotary_dim, flags, mscale, stream);
}

int fa_page_plan(const int* lens, const int* new_lens, int* table, int table_width, int* queue,
                 int queue_size, const int* queue_state, int B, int page_size, int num_tokens,
                 int* lens_out, int* q_offsets, int* positions, int* slots, int* queue_state_out,
                 void* stream) {
  if (!lens || !new_lens || !table || !queue || !queue_state || !lens_out || !q_offsets ||
      !queue_state_out)
    return FA_ERR_INVALID_ARG;
  if (B < 1 || table_width < 1 || queue_size < 1 || num_tokens < 0) return FA_ERR_INVALID_ARG;
  if (num_tokens > 0 && (!positions || !slots)) return FA_ERR_INVALID_ARG;
  // other thread blocks read the old lengths and state while the new ones are written
  if (lens_out == lens || lens_out == new_lens || queue_state_out == queue_state)
    return FA_ERR_INVALID_ARG;
  if (B > kPlanMaxBatch || !page_size_ok(page_size) || !width_ok(table_width, page_size) ||
      static_cast<long long>(B) * table_width > 0x7fffffffll)
    return FA_ERR_UNSUPPORTED;
  for (const void* p : {static_cast<const void*>(lens), static_cast<const void*>(new_lens),
                        static_cast<const void*>(table), static_cast<const void*>(queue),
                        static_cast<const void*>(queue_state), static_cast<const void*>(lens_out),
                        static_cast<const void*>(q_offsets), static_cast<const void*>(positions),
                        static_cast<const void*>(slots), static_cast<const void*>(queue_state_out)})
    if (!aligned(p, 4)) return FA_ERR_MISALIGNED;
  PlanArgs a{lens,     new_lens,  table, queue,           queue_state, lens_out,   q_offsets,
             positions, slots,    queue_state_out, B,     table_width, queue_size,
             log2_of(page_size), num_tokens};
  const int smem = (3 * B + 1) * 4;
  static std::atomic<uint64_t> done{0};
  if (int rc = opt_in_smem(page_plan_kernel, (3 * kPlanMaxBatch + 1) * 4, done)) return rc;
  // a warp per request and a thread per token, one CTA a SM at most: each repeats the scan over the
  // lengths (1000 requests, 46,000 tokens, some ended: 9.4 us; 15.8 with four tokens a thread on a quarter of
  // the CTAs; a single CTA for a small step: 2.9 us)
  const long long items = num_tokens > 32ll * B ? num_tokens : 32ll * B;
  long long grid = (items + kPlanThreads - 1) / kPlanThreads;
  if (grid > kSms) grid = kSms;
  return launch_early(page_plan_kernel, static_cast<unsigned>(grid), kPlanThreads, smem,
                static_cast<cudaStream_t>(stream), a);
}

size_t fa_kv4_cache_bytes(int num_pages, int Hkv, int page_size, int d) {
  if (num_pages < 1 || Hkv < 1 || Hkv > 65535 || !page_size_ok(page_size) || (d != 64 && d != 128)) return 0;
  if (static_cast<long long>(num_pages) * page_size > 0x7fffffffll) return 0;
  return static_cast<size_t>(num_pages) * Hkv * 2 * kv4_block_bytes(page_size, d);
}

int fa_kv4_append(const void* k, long long k_row_stride, long long k_head_stride, const void* v,
                  long long v_row_stride, long long v_head_stride, void* cache, int num_pages,
                  int page_size, const int* slots, int T, int Hkv, int d, float k_descale,
                  float v_descale, void* stream) {
  if (!k || !v || !slots || T < 1) return FA_ERR_INVALID_ARG;
  if (k_row_stride < 0 || k_head_stride < 0 || v_row_stride < 0 || v_head_stride < 0)
    return FA_ERR_INVALID_ARG;
  if (!power_of_two(k_descale) || !power_of_two(v_descale)) return FA_ERR_INVALID_ARG;
  if (int rc = cache_checks(cache, num_pages, Hkv, page_size, d)) return rc;
  if (k_row_stride % 8 || k_head_stride % 8 || v_row_stride % 8 || v_head_stride % 8 ||
      !aligned(k, 16) || !aligned(v, 16) || !aligned(slots, 4))
    return FA_ERR_MISALIGNED;
  Kv4Rows a{};
  a.in[0] = static_cast<const __nv_bfloat16*>(k);
  a.in[1] = static_cast<const __nv_bfloat16*>(v);
  a.cache = static_cast<uint8_t*>(cache);
  a.slots = slots;
  a.row[0] = k_row_stride;
  a.head[0] = k_head_stride;
  a.row[1] = v_row_stride;
  a.head[1] = v_head_stride;
  a.heads = Hkv;
  a.page_shift = log2_of(page_size);
  a.pages = num_pages;
  a.descale[0] = k_descale;
  a.descale[1] = v_descale;
  return launch_rows(a, T, Hkv, d, kKv4Group, kv4_append_kernel<64>, kv4_append_kernel<128>,
                     static_cast<cudaStream_t>(stream));
}

int fa_kv4_read(const void* cache, int num_pages, int page_size, const int* slots, void* k, void* v,
                int T, int Hkv, int d, float k_descale, float v_descale, void* stream) {
  if (!k || !v || k == v || !slots || T < 1) return FA_ERR_INVALID_ARG;
  if (!power_of_two(k_descale) || !power_of_two(v_descale)) return FA_ERR_INVALID_ARG;
  if (int rc = cache_checks(cache, num_pages, Hkv, page_size, d)) return rc;
  if (!aligned(k, 16) || !aligned(v, 16) || !aligned(slots, 4)) return FA_ERR_MISALIGNED;
  Kv4Rows a{};
  a.out[0] = static_cast<__nv_bfloat16*>(k);
  a.out[1] = static_cast<__nv_bfloat16*>(v);
  a.cache = static_cast<uint8_t*>(const_cast<void*>(cache));
  a.slots = slots;
  a.heads = Hkv;
  a.page_shift = log2_of(page_size);
  a.pages = num_pages;
  a.descale[0] = k_descale;
  a.descale[1] = v_descale;
  return launch_rows(a, T, Hkv, d, 8, kv4_read_kernel<64>, kv4_read_kernel<128>,
                     static_cast<cudaStream_t>(stream));
}

size_t fa_kv4_fwd_workspace_bytes(int Hq, int Hkv, int d, int max_q, int page_size,
                                  int table_width) {
  if (Hq < 1 || Hkv < 1 || Hq % Hkv || max_q < 1 || (d != 64 && d != 128)) return 0;
  if (!page_size_ok(page_size) || table_width < 1 || !width_ok(table_width, page_size)) return 0;
  const int nt = dec_row_eights(static_cast<long long>(max_q) * (Hq / Hkv));
  return nt && dec_whole_tiles(d, nt, page_size, table_width) ? 0 : kv4_workspace(nt, d);
}

int fa_kv4_fwd(const void* q, long long q_row_stride, long long q_head_stride, const void* cache,
               int num_pages, int page_size, const int* table, int table_width, const int* lens,
               const int* q_offsets, void* o, float* lse, int T, int B, int Hq, int Hkv, int d,
               int max_q, float scale, int causal, float k_descale, float v_descale,
               void* workspace, size_t workspace_bytes, int* dev_status, void* stream) {
  if (!q || !table || !lens || !o || !lse || o == q) return FA_ERR_INVALID_ARG;
  if (T < 1 || B < 1 || Hq < 1 || Hkv < 1 || Hq % Hkv || table_width < 1 || max_q < 1)
    return FA_ERR_INVALID_ARG;
  if (!q_offsets && T % B) return FA_ERR_INVALID_ARG;
  if (q_row_stride < 0 || q_head_stride < 0) return FA_ERR_INVALID_ARG;
  if (!std::isfinite(scale) || scale < 0.f) return FA_ERR_INVALID_ARG;
  if (!power_of_two(k_descale) || !power_of_two(v_descale)) return FA_ERR_INVALID_ARG;
  if (int rc = cache_checks(cache, num_pages, Hkv, page_size, d)) return rc;
  if (static_cast<long long>(T) * Hq > 0x3fffffffll || !width_ok(table_width, page_size))
    return FA_ERR_UNSUPPORTED;
  const int nt = dec_row_eights(static_cast<long long>(max_q) * (Hq / Hkv));
  const int whole = nt ? dec_whole_tiles(d, nt, page_size, table_width) : 0;
  if (!whole && (!workspace || workspace_bytes < kv4_workspace(nt, d))) return FA_ERR_INVALID_ARG;
  if (q_row_stride % 8 || q_head_stride % 8 || !aligned(q, 16) || !aligned(o, 16) ||
      !aligned(lse, 4) || !aligned(table, 4) || !aligned(lens, 4) || !aligned(q_offsets, 4) ||
      !aligned(workspace, 16) || !aligned(dev_status, 4))
    return FA_ERR_MISALIGNED;
  const double c = static_cast<double>(scale) * 1.4426950408889634 * k_descale;
  if (!(c <= 3.0e38)) return FA_ERR_INVALID_ARG;
  Kv4Args a{};
  a.q = static_cast<const __nv_bfloat16*>(q);
  a.q_row = q_row_stride;
  a.q_head = q_head_stride;
  a.cache = static_cast<const uint8_t*>(cache);
  a.table = table;
  a.lens = lens;
  a.q_offsets = q_offsets;
  a.o = static_cast<__nv_bfloat16*>(o);
  a.lse = lse;
  a.q_len = T / B;
  a.t = T;
  a.b = B;
  a.hq = Hq;
  a.hk = Hkv;
  a.group = Hq / Hkv;
  a.width = table_width;
  a.page_shift = log2_of(page_size);
  a.pages = num_pages;
  a.causal = causal != 0;
  a.whole_tiles = whole;
  a.c = static_cast<float>(c);
  a.v_descale = v_descale;
  a.status = dev_status;
  if (!a.status && nt == 0) {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxKvDevices) return FA_ERR_CUDA;
    a.status = library_status_ptr(dev);
    if (!a.status) return FA_ERR_CUDA;
  }
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return d == 64 ? launch_kv4<64>(a, nt, workspace, s) : launch_kv4<128>(a, nt, workspace, s);
}

int fa_kv4_move(void* const* caches, int num_caches, int num_pages, int page_size, int Hkv, int d, const int* sources,
                const int* slots, const int* q_offsets, const int* counts, int T, int B, void* stream) {
  if (!caches || !sources || !slots || !q_offsets || !counts || num_caches < 1 || T < 1 || B < 1)
    return FA_ERR_INVALID_ARG;
  if (num_caches > kMoveLayers) return FA_ERR_UNSUPPORTED;
  if (!aligned(sources, 4) || !aligned(slots, 4) || !aligned(q_offsets, 4) || !aligned(counts, 4))
    return FA_ERR_MISALIGNED;
  Kv4MoveArgs a{};
  for (int i = 0; i < num_caches; ++i) {
    if (int rc = cache_checks(caches[i], num_pages, Hkv, page_size, d)) return rc;
    a.cache[i] = static_cast<uint8_t*>(caches[i]);
  }
  a.sources = sources;
  a.slots = slots;
  a.offsets = q_offsets;
  a.counts = counts;
  a.t = T;
  a.b = B;
  a.heads = Hkv;
  a.page_shift = log2_of(page_size);
  a.pages = num_pages;
  const long long pieces = 18ll * Hkv * B;  // threads of a cache
  if (pieces > 0x7fffffffll - kKv4Threads) return FA_ERR_UNSUPPORTED;
  const dim3 grid(static_cast<unsigned>((pieces + kKv4Threads - 1) / kKv4Threads), static_cast<unsigned>(num_caches));
  return launch_early(d == 64 ? kv4_move_kernel<64> : kv4_move_kernel<128>, grid, kKv4Threads, 0,
                      static_cast<cudaStream_t>(stream), a);
}

}  // extern "C"
