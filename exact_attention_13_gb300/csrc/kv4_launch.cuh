// kv4_launch.cuh -- launches of the attention kernels over the 4-bit cache, which the host sides of kv4_fwd and
// kv4_tree_fwd share.
#pragma once

#include "kv4_attn.cuh"
#include "kv4_chunk.cuh"
#include "kv_host.cuh"

namespace exattn {

namespace {

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

template <int D, int NT, bool TREE = false>
int launch_decode(Kv4Args& a, void* workspace, cudaStream_t s) {
  constexpr int n = kv4_ctas(NT);
  if (!a.whole_tiles) split_workspace<D, NT>(a, workspace);
  constexpr int smem = dec_smem_bytes<D, NT>();
  static_assert(dec_ctas_per_sm(NT) * (smem + 2048) <= 228 * 1024, "shared memory per SM");
  static std::atomic<uint64_t> done{0};
  auto kern = kv4_decode_kernel<D, NT, TREE>;
  if (int rc = opt_in_smem(kern, smem, done)) return rc;
  kern<<<n, kDecThreads, smem, s>>>(a);
  if (int rc = launched()) return rc;
  if (a.whole_tiles) return FA_OK;
  static_assert(n <= 2 * kMergeThreads && 2 * n <= 0x7fff, "descriptors of the merge");
  return launch_merge<D, 8 * NT>(a, n, s);
}

template <int D, bool TREE = false>
int launch_chunk(Kv4Args& a, void* workspace, cudaStream_t s) {
  constexpr int n = kv4_ctas(0);
  split_workspace<D, 0>(a, workspace);
  constexpr int smem = chunk_smem_bytes<D>();
  // more than half of an SM's, so that one CTA (with all of the tensor memory) runs there
  static_assert(smem <= 227 * 1024 && smem > 114 * 1024, "shared memory per CTA");
  static std::atomic<uint64_t> done{0};
  auto kern = kv4_chunk_kernel<D, TREE>;
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

}  // namespace
}  // namespace exattn
