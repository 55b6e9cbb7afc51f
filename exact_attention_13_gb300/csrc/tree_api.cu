// tree_api.cu -- host side of trees of drafted tokens: their plan, attention over the 4-bit cache and acceptance.
// Argument checks and launches of the C ABI declared in include/exact_attention.h; no call allocates, synchronises
// or throws.
#include <cuda_runtime.h>

#include <atomic>
#include <cmath>
#include <cstdint>
#include <initializer_list>

#include "../../include/exact_attention.h"
#include "kv4_launch.cuh"
#include "kv4_tree.cuh"
#include "kv_host.cuh"
#include "tree_plan.cuh"

namespace exattn {

namespace {

// The kernel for `rows` query rows of a key head: 8 or 16 (kv4_attn.cuh, every value widened in registers), units of 32
// or 64 (kv4_tree.cuh) or of 256 (kv4_chunk.cuh).  Both sides of each border in us, the chosen one first, for 64
// requests of 4096 keys, 8 key heads, d 128: 8 rows 67 by the 8s, 89 by the 16s; 16 rows 91, 118 by the 32s; 32 rows 123,
// 142 by the 64s (two 16s: 169); 64 rows 141, 210 by 256; 128 rows 214 by 256, 271 by two 64s (with 500 to 8192 keys
// 248 and 296).  Where a third of the requests fits one 64 the two are alike: 40 to 128 rows 212 and 222.  Only this
// load and d 128 have both sides measured; for few requests or d 64 the rule is the same and its borders are not shown.
int tree_rows(long long rows) { return rows <= 8 ? 8 : rows <= 16 ? 16 : rows <= 32 ? 32 : rows <= 64 ? 64 : 256; }

size_t tree_workspace(int n, int d) {
  if (n <= 16) return kv4_workspace(n / 8, d);
  if (n == 256) return kv4_workspace(0, d);
  const size_t rows = static_cast<size_t>(2) * kSms * n;
  return (rows * (d * 4 + 8) + kSms * 16 + 255) / 256 * 256;
}

// Tables of at most this many tiles: units are not split, which saves the merge kernel and the workspace.
constexpr int kTreeWholeTiles = 4;
int tree_whole_tiles(int n, int d, int page, int width) {
  if (n <= 16) return dec_whole_tiles(d, n / 8, page, width);
  const long long tiles = (static_cast<long long>(page) * width + kTrKeys - 1) / kTrKeys;
  return n < 256 && tiles <= kTreeWholeTiles ? static_cast<int>(tiles) : 0;
}

template <int D, int N>
int launch_tree(Kv4Args& a, void* workspace, cudaStream_t s) {
  if (!a.whole_tiles) {
    constexpr size_t rows = static_cast<size_t>(2) * kSms * N;
    a.part_o = static_cast<float*>(workspace);
    a.part_ml = reinterpret_cast<float2*>(a.part_o + rows * D);
    a.desc = reinterpret_cast<int4*>(a.part_ml + rows);
  }
  constexpr int smem = tree_smem_bytes<D, N>();
  // more than half of an SM's, so that one CTA (with all of the tensor memory) runs there
  constexpr int taken = smem > 120 * 1024 ? smem : 120 * 1024;
  static_assert(smem <= 227 * 1024, "shared memory per CTA");
  static std::atomic<uint64_t> done{0};
  auto kern = kv4_tree_kernel<D, N>;
  if (!done.load(std::memory_order_acquire)) {
    // a build with fewer registers at launch would wait forever for the ones to redistribute
    cudaFuncAttributes attr;
    if (cudaFuncGetAttributes(&attr, kern) != cudaSuccess) return FA_ERR_CUDA;
    if (attr.numRegs < kTrLaunchRegs) return FA_ERR_UNSUPPORTED;
  }
  if (int rc = opt_in_smem(kern, taken, done)) return rc;
  kern<<<kSms, kTrThreads, taken, s>>>(a);
  if (int rc = launched()) return rc;
  return a.whole_tiles ? FA_OK : launch_merge<D, N>(a, kSms, s);
}

template <int D>
int launch_tree_rows(Kv4Args& a, int n, void* workspace, cudaStream_t s) {
  return n == 8     ? launch_decode<D, 1, true>(a, workspace, s)
         : n == 16  ? launch_decode<D, 2, true>(a, workspace, s)
         : n == 32  ? launch_tree<D, 32>(a, workspace, s)
         : n == 64  ? launch_tree<D, 64>(a, workspace, s)
                    : launch_chunk<D, true>(a, workspace, s);
}

}  // namespace
}  // namespace exattn

using namespace exattn;

extern "C" {

int fa_tree_plan(const int* parents, const int* q_offsets, const int* lens, int B, int T, int words, int* positions,
                 unsigned* seen, void* stream) {
  if (!parents || !q_offsets || !lens || !positions || !seen || B < 1 || T < 1 || words < 1) return FA_ERR_INVALID_ARG;
  if (words > kTreeWords || B > kPlanMaxBatch || static_cast<long long>(T) * words > 0x7fffffffll)
    return FA_ERR_UNSUPPORTED;
  for (const void* p : {static_cast<const void*>(parents), static_cast<const void*>(q_offsets),
                        static_cast<const void*>(lens), static_cast<const void*>(positions),
                        static_cast<const void*>(seen)})
    if (!aligned(p, 4)) return FA_ERR_MISALIGNED;
  const TreePlanArgs a{parents, q_offsets, lens, positions, seen, B, T, words};
  return launch_early(tree_plan_kernel, static_cast<unsigned>(B + 1), kTreeThreads, 0,
                      static_cast<cudaStream_t>(stream), a);
}

int fa_tree_accept(const int* parents, const unsigned* seen, int words, const int* tokens, const int* choices,
                   const int* lens, const int* new_lens, const int* q_offsets, const int* slots, const int* table,
                   int table_width, int* queue, int queue_size, const int* queue_state, int B, int page_size, int T,
                   int* lens_out, int* counts, int* path, int* next_tokens, int* sources, int* queue_state_out,
                   void* stream) {
  if (!lens || !new_lens || !q_offsets || !table || !queue || !queue_state || !lens_out || !counts || !next_tokens ||
      !queue_state_out)
    return FA_ERR_INVALID_ARG;
  if (T > 0 && (!parents || !seen || !tokens || !choices || !slots || !path || !sources)) return FA_ERR_INVALID_ARG;
  if (B < 1 || T < 0 || words < 1 || table_width < 1 || queue_size < 1) return FA_ERR_INVALID_ARG;
  // other thread blocks, and the second kernel, read the old lengths and state
  if (lens_out == lens || lens_out == new_lens || queue_state_out == queue_state) return FA_ERR_INVALID_ARG;
  if (words > kTreeWords || B > kPlanMaxBatch || !page_size_ok(page_size) || !width_ok(table_width, page_size) ||
      static_cast<long long>(B) * table_width > 0x7fffffffll || static_cast<long long>(T) * words > 0x7fffffffll)
    return FA_ERR_UNSUPPORTED;
  for (const void* p : {static_cast<const void*>(parents), static_cast<const void*>(seen),
                        static_cast<const void*>(tokens), static_cast<const void*>(choices),
                        static_cast<const void*>(lens), static_cast<const void*>(new_lens),
                        static_cast<const void*>(q_offsets), static_cast<const void*>(slots),
                        static_cast<const void*>(table), static_cast<const void*>(queue),
                        static_cast<const void*>(queue_state), static_cast<const void*>(lens_out),
                        static_cast<const void*>(counts), static_cast<const void*>(path),
                        static_cast<const void*>(next_tokens), static_cast<const void*>(sources),
                        static_cast<const void*>(queue_state_out)})
    if (!aligned(p, 4)) return FA_ERR_MISALIGNED;
  const TreeAcceptArgs a{parents, seen,   tokens, choices,     lens,     new_lens,        q_offsets, slots,
                         table,   queue,  queue_state, lens_out, counts, path,            next_tokens, sources,
                         queue_state_out, B,      T,      words,       table_width, queue_size, log2_of(page_size)};
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (B <= kTreeGroups * kTreeCluster) {
    const unsigned n = static_cast<unsigned>((B + kTreeGroups - 1) / kTreeGroups);
    return launch_early_clusters(n, tree_accept_small_kernel, n, kTreeGroups * kTreeThreads, 0, s, a);
  }
  if (int rc = launch_early(tree_accept_kernel, static_cast<unsigned>(B + 1), kTreeThreads, 0, s, a)) return rc;
  static std::atomic<uint64_t> done{0};
  if (int rc = opt_in_smem(tree_release_kernel, kPlanMaxBatch * 4, done)) return rc;
  long long grid = (32ll * B + kPlanThreads - 1) / kPlanThreads;  // a warp a request
  if (grid > kSms) grid = kSms;
  return launch_early(tree_release_kernel, static_cast<unsigned>(grid), kPlanThreads, B * 4, s, a);
}

size_t fa_kv4_tree_fwd_workspace_bytes(int Hq, int Hkv, int d, int max_q, int page_size, int table_width) {
  if (Hq < 1 || Hkv < 1 || Hq % Hkv || max_q < 1 || (d != 64 && d != 128)) return 0;
  if (!page_size_ok(page_size) || table_width < 1 || !width_ok(table_width, page_size)) return 0;
  const int n = tree_rows(static_cast<long long>(max_q) * (Hq / Hkv));
  return tree_whole_tiles(n, d, page_size, table_width) ? 0 : tree_workspace(n, d);
}

int fa_kv4_tree_fwd(const void* q, long long q_row_stride, long long q_head_stride, const void* cache, int num_pages,
                    int page_size, const int* table, int table_width, const int* lens, const int* q_offsets,
                    const unsigned* seen, int words, void* o, float* lse, int T, int B, int Hq, int Hkv, int d,
                    int max_q, float scale, float k_descale, float v_descale, void* workspace, size_t workspace_bytes,
                    int* dev_status, void* stream) {
  if (!q || !table || !lens || !q_offsets || !seen || !o || !lse || o == q) return FA_ERR_INVALID_ARG;
  if (T < 1 || B < 1 || Hq < 1 || Hkv < 1 || Hq % Hkv || table_width < 1 || max_q < 1 || words < 1)
    return FA_ERR_INVALID_ARG;
  if (q_row_stride < 0 || q_head_stride < 0) return FA_ERR_INVALID_ARG;
  if (!std::isfinite(scale) || scale < 0.f) return FA_ERR_INVALID_ARG;
  if (!power_of_two(k_descale) || !power_of_two(v_descale)) return FA_ERR_INVALID_ARG;
  if (int rc = cache_checks(cache, num_pages, Hkv, page_size, d)) return rc;
  if (static_cast<long long>(T) * Hq > 0x3fffffffll || !width_ok(table_width, page_size) || words > kTreeWords)
    return FA_ERR_UNSUPPORTED;
  const int n = tree_rows(static_cast<long long>(max_q) * (Hq / Hkv)), whole = tree_whole_tiles(n, d, page_size, table_width);
  if (!whole && (!workspace || workspace_bytes < tree_workspace(n, d))) return FA_ERR_INVALID_ARG;
  if (q_row_stride % 8 || q_head_stride % 8 || !aligned(q, 16) || !aligned(o, 16) || !aligned(lse, 4) ||
      !aligned(table, 4) || !aligned(lens, 4) || !aligned(q_offsets, 4) || !aligned(seen, 4) ||
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
  a.t = T;
  a.b = B;
  a.hq = Hq;
  a.hk = Hkv;
  a.group = Hq / Hkv;
  a.width = table_width;
  a.page_shift = log2_of(page_size);
  a.pages = num_pages;
  a.whole_tiles = whole;
  a.c = static_cast<float>(c);
  a.v_descale = v_descale;
  a.tree = seen;
  a.words = words;
  a.status = dev_status;
  if (!a.status && n > 16) {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxKvDevices) return FA_ERR_CUDA;
    a.status = library_status_ptr(dev);
    if (!a.status) return FA_ERR_CUDA;
  }
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return d == 64 ? launch_tree_rows<64>(a, n, workspace, s) : launch_tree_rows<128>(a, n, workspace, s);
}

}  // extern "C"
