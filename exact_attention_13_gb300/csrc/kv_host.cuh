// kv_host.cuh -- argument checks and launches that the host sides of the operators around attention share.
#pragma once

#include <cuda_runtime.h>

#include <atomic>
#include <cmath>
#include <cstdint>

#include "../../include/exact_attention.h"

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

// Launch a kernel that may begin while the one before it on the stream still runs (grid_wait in each), in clusters of
// `cluster` CTAs.
template <typename... Params, typename... Args>
int launch_early_clusters(unsigned cluster, void (*kern)(Params...), dim3 grid, int threads, int smem, cudaStream_t s,
                          const Args&... args) {
  cudaLaunchConfig_t config{};
  config.gridDim = grid;
  config.blockDim = dim3(threads);
  config.dynamicSmemBytes = smem;
  config.stream = s;
  cudaLaunchAttribute attrs[2]{};
  attrs[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attrs[0].val.programmaticStreamSerializationAllowed = 1;
  attrs[1].id = cudaLaunchAttributeClusterDimension;
  attrs[1].val.clusterDim.x = cluster;
  attrs[1].val.clusterDim.y = attrs[1].val.clusterDim.z = 1;
  config.attrs = attrs;
  config.numAttrs = cluster > 1 ? 2 : 1;
  if (cudaLaunchKernelEx(&config, kern, args...) == cudaSuccess) return FA_OK;
  (void)cudaGetLastError();
  return FA_ERR_CUDA;
}

template <typename... Params, typename... Args>
int launch_early(void (*kern)(Params...), dim3 grid, int threads, int smem, cudaStream_t s, const Args&... args) {
  return launch_early_clusters(1, kern, grid, threads, smem, s, args...);
}

int cache_checks(const void* cache, int pages, int heads, int page, int d) {
  if (!cache || pages < 1 || heads < 1) return FA_ERR_INVALID_ARG;
  if ((d != 64 && d != 128) || !page_size_ok(page) || heads > 65535) return FA_ERR_UNSUPPORTED;
  if (static_cast<long long>(pages) * page > 0x7fffffffll) return FA_ERR_UNSUPPORTED;
  return aligned(cache, 16) ? FA_OK : FA_ERR_MISALIGNED;
}

}  // namespace
}  // namespace exattn
