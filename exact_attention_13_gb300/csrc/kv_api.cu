// kv_api.cu -- host side of the operators around attention: rotary positions, page planning, the
// 4-bit key/value cache and attention over it.  Argument checks and launches of the C ABI declared
// in include/exact_attention.h; no call allocates, synchronises or throws.
#include <cuda_runtime.h>

#include <atomic>
#include <cmath>
#include <cstdint>
#include <initializer_list>

#include "../../include/exact_attention.h"
#include "kv4_attn.cuh"
#include "kv4_cache.cuh"
#include "kv4_chunk.cuh"
#include "page_plan.cuh"
#include "rope.cuh"

namespace exattn {

int* library_status_ptr(int dev);  // fa_api.cu

namespace {

constexpr int kSms = 152;
constexpr int kMaxKvDevices = 64;

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

bool power_of_two(float x) {
  if (!(x > 0.f) || !std::isfinite(x)) return false;
  int e = 0;
  return std::frexp(x, &e) == 0.5f && e >= -60 && e <= 60;
}

bool page_size_ok(int page) { return page == 16 || page == 32 || page == 64 || page == 128; }

// Tokens of one row of a page table: tiles and strips past the last one are still 32-bit numbers.
bool width_ok(int width, int page) { return static_cast<long long>(width) * page <= 1ll << 30; }

int log2_of(int x) {
  int s = 0;
  while ((1 << s) < x) ++s;
  return s;
}

int launched() { return cudaGetLastError() == cudaSuccess ? FA_OK : FA_ERR_CUDA; }

// Set an attribute of a kernel, once per device.
template <typename K>
int set_once(K kern, cudaFuncAttribute attribute, int value, std::atomic<uint64_t>& done) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxKvDevices) return FA_ERR_CUDA;
  if (done.load(std::memory_order_acquire) & (1ull << dev)) return FA_OK;
  if (cudaFuncSetAttribute(kern, attribute, value) != cudaSuccess) return FA_ERR_CUDA;
  done.fetch_or(1ull << dev, std::memory_order_acq_rel);
  return FA_OK;
}

template <typename K>
int opt_in_smem(K kern, int bytes, std::atomic<uint64_t>& done) {
  return set_once(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes, done);
}

// Launch a kernel that may begin while the one before it on the stream still runs (grid_wait in each).
template <typename... Params, typename... Args>
int launch_early(void (*kern)(Params...), dim3 grid, int threads, int smem, cudaStream_t s, const Args&... args) {
  cudaLaunchConfig_t config{};
  config.gridDim = grid;
  config.blockDim = dim3(threads);
  config.dynamicSmemBytes = smem;
  config.stream = s;
  cudaLaunchAttribute early{};
  early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  early.val.programmaticStreamSerializationAllowed = 1;
  config.attrs = &early;
  config.numAttrs = 1;
  if (cudaLaunchKernelEx(&config, kern, args...) == cudaSuccess) return FA_OK;
  (void)cudaGetLastError();
  return FA_ERR_CUDA;
}

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

// ---------------------------------------------------------------------------------- cache
int cache_checks(const void* cache, int pages, int heads, int page, int d) {
  if (!cache || pages < 1 || heads < 1) return FA_ERR_INVALID_ARG;
  if ((d != 64 && d != 128) || !page_size_ok(page) || heads > 65535) return FA_ERR_UNSUPPORTED;
  if (static_cast<long long>(pages) * page > 0x7fffffffll) return FA_ERR_UNSUPPORTED;
  return aligned(cache, 16) ? FA_OK : FA_ERR_MISALIGNED;
}

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
// CTAs of one SM, by eights of rows of a unit: up to 168 registers a thread beside eight rows, 255
// beside more.  (16 rows with three CTAs: 60 us instead of 50 for 16 requests of 15 rows, 57 with strips
// of 16 keys; 8 rows with four: no gain.)
constexpr int dec_ctas_per_sm(int nt) { return nt == 1 ? 3 : 2; }

// Query rows that share a unit, in eights: the smallest of 8, 16 and 32 that hold the rows of one
// key head (fewer padded rows); 0 for more rows than that: the kernel for prompt chunks.
int dec_row_eights(long long rows) { return rows <= 8 ? 1 : rows <= 16 ? 2 : rows <= 32 ? 4 : 0; }

// CTAs and rows of a unit of the kernel for `nt` eights of rows, and its workspace.
constexpr int kv4_ctas(int nt) { return nt ? kSms * dec_ctas_per_sm(nt) : kSms; }
constexpr size_t kv4_part_rows(int nt) {
  return static_cast<size_t>(2) * kv4_ctas(nt) * (nt ? 8 * nt : kChRows);
}
size_t kv4_workspace(int nt, int d) {
  return (kv4_part_rows(nt) * (d * 4 + 8) + kv4_ctas(nt) * 16 + 255) / 256 * 256;
}

// Tables of at most this many tiles: units are not split, which saves the merge kernel and the
// workspace; a unit's tiles then run one after the other.
constexpr int kWholeTiles = 4;
int dec_whole_tiles(int d, int nt, int page, int width) {
  const int tile = d == 64 ? dec_tile<64, 8>() : nt == 4 ? dec_tile<128, 32>() : dec_tile<128, 8>();
  const long long tiles = (static_cast<long long>(page) * width + tile - 1) / tile;
  return tiles <= kWholeTiles ? static_cast<int>(tiles) : 0;
}

template <int D, int NT>
void split_workspace(Kv4Args& a, void* workspace) {
  a.part_o = static_cast<float*>(workspace);
  a.part_ml = reinterpret_cast<float2*>(a.part_o + kv4_part_rows(NT) * D);
  a.desc = reinterpret_cast<int4*>(a.part_ml + kv4_part_rows(NT));
}

template <int D, int R>
int launch_merge(const Kv4Args& a, int ctas, cudaStream_t s) {
  // Few units (at most one for eight CTAs): each may span many CTAs, and rows get blocks of their own
  // (4 units of 8 rows in 114 parts each: 3.9 us instead of 7 with blocks for all CTAs; 128 units of 15
  // rows: 2.4 us more than the other way).  Else eight rows a block, 64 of a prompt chunk (135 us
  // for the whole call of 4 chunks of 512 tokens; 139 with eight).
  const bool few = static_cast<long long>(a.b) * a.hk <= ctas / 8;
  const dim3 grid = few ? dim3(ctas / 8, R > 32 ? 32 : R) : dim3(ctas, R > 32 ? R / 64 : R / 8);
  return launch_early(kv4_merge_kernel<D, R>, grid, kMergeThreads, 0, s, a, few ? ctas : 0);
}

template <int D, int NT>
int launch_decode(Kv4Args& a, void* workspace, cudaStream_t s) {
  constexpr int n = kv4_ctas(NT);
  if (!a.whole_tiles) split_workspace<D, NT>(a, workspace);
  constexpr int smem = dec_smem_bytes<D, NT>();
  static_assert(dec_ctas_per_sm(NT) * (smem + 2048) <= 228 * 1024, "shared memory per SM");
  static std::atomic<uint64_t> done{0};
  auto kern = kv4_decode_kernel<D, NT>;
  if (int rc = opt_in_smem(kern, smem, done)) return rc;
  kern<<<n, kDecThreads, smem, s>>>(a);
  if (int rc = launched()) return rc;
  if (a.whole_tiles) return FA_OK;
  static_assert(n <= 2 * kMergeThreads && 2 * n <= 0x7fff, "descriptors of the merge");
  return launch_merge<D, 8 * NT>(a, n, s);
}

template <int D>
int launch_chunk(Kv4Args& a, void* workspace, cudaStream_t s) {
  constexpr int n = kv4_ctas(0);
  split_workspace<D, 0>(a, workspace);
  constexpr int smem = chunk_smem_bytes<D>();
  // more than half of an SM's, so that one CTA (with all of the tensor memory) runs there
  static_assert(smem <= 227 * 1024 && smem > 114 * 1024, "shared memory per CTA");
  static std::atomic<uint64_t> done{0};
  auto kern = kv4_chunk_kernel<D>;
  if (!done.load(std::memory_order_acquire)) {
    // a build with fewer registers at launch would wait forever for the ones to redistribute
    cudaFuncAttributes attr;
    if (cudaFuncGetAttributes(&attr, kern) != cudaSuccess) return FA_ERR_CUDA;
    if (attr.numRegs < kChLaunchRegs) return FA_ERR_UNSUPPORTED;
  }
  if (int rc = opt_in_smem(kern, smem, done)) return rc;
  kern<<<n, kChThreads, smem, s>>>(a);
  if (int rc = launched()) return rc;
  return launch_merge<D, kChRows>(a, n, s);
}

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
  if (!positions || !turns || B < 1 || N < 1 || Hq < 1 || Hk < 0 || positions_batch_stride < 0)
    return FA_ERR_INVALID_ARG;
  if (flags & ~(FA_ROPE_INTERLEAVED | FA_ROPE_INVERSE)) return FA_ERR_INVALID_ARG;
  if (!std::isfinite(mscale)) return FA_ERR_INVALID_ARG;
  if (d != 64 && d != 128) return FA_ERR_UNSUPPORTED;
  if (rotary_dim < 16 || rotary_dim > d || rotary_dim % 16) return FA_ERR_UNSUPPORTED;
  if (!aligned(positions, 4) || !aligned(turns, 8)) return FA_ERR_MISALIGNED;
  RopeArgs a;
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
  auto kern = il ? inv ? rope_kernel<true, true> : rope_kernel<true, false>
                 : inv ? rope_kernel<false, true> : rope_kernel<false, false>;
  return launch_early(kern, grid, kRopeThreads, 0, s, a);
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

}  // extern "C"
