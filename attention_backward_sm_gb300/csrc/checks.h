// Checks of arguments that the C entry points of the operators around the
// cache share.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>

#include "../../include/fabwd.h"
#include "internal.h"
#include "paged.h"

namespace fa {

inline int ok() { return set_last_error(FA_OK, "%s", ""); }

inline int cuda_fail(cudaError_t e, const char* where) {
  return set_last_error(FA_ERR_CUDA, "%s: %s (%s)", where, cudaGetErrorName(e), cudaGetErrorString(e));
}

inline bool misaligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) != 0; }
inline bool misaligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) != 0; }

// The current device, which has to be what the library is built for.
inline int check_device(Device& d) {
  static std::atomic<int> known[64];   // SMs of the devices already found to be sm_103
  cudaError_t e = cudaGetDevice(&d.id);
  if (e != cudaSuccess) return cuda_fail(e, "cudaGetDevice");
  const bool listed = d.id >= 0 && d.id < 64;
  d.sms = listed ? known[d.id].load(std::memory_order_acquire) : 0;
  if (d.sms > 0) return FA_OK;
  int major = 0, minor = 0;
  cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, d.id);
  cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, d.id);
  if (major != 10 || minor != 3)
    return set_last_error(FA_ERR_UNSUPPORTED, "this library is built for sm_103a; device %d is sm_%d%d", d.id, major,
                          minor);
  e = cudaDeviceGetAttribute(&d.sms, cudaDevAttrMultiProcessorCount, d.id);
  if (e != cudaSuccess) return cuda_fail(e, "cudaDeviceGetAttribute");
  if (listed) known[d.id].store(d.sms, std::memory_order_release);
  return FA_OK;
}

// The cache's sizes, strides and types; pointers only where they are set.
inline int check_cache(const PagedCache& c, int kv_type) {
  if (kv_type != FA_KV_BF16 && kv_type != FA_KV_E4M3)
    return set_last_error(FA_ERR_INVALID_ARG, "kv_type must be 0 (bf16) or 1 (e4m3), got %d", kv_type);
  if (c.head_dim != 64 && c.head_dim != 128 && c.head_dim != 256)
    return set_last_error(FA_ERR_UNSUPPORTED, "head_dim must be 64, 128 or 256, got %d", c.head_dim);
  if (c.heads_kv < 1) return set_last_error(FA_ERR_INVALID_ARG, "heads_kv must be >= 1, got %d", c.heads_kv);
  if (c.num_pages < 0) return set_last_error(FA_ERR_INVALID_ARG, "num_pages must be >= 0, got %d", c.num_pages);
  if (c.page_size < 1) return set_last_error(FA_ERR_INVALID_ARG, "page_size must be >= 1, got %d", c.page_size);
  if (kv_type == FA_KV_BF16 && (c.k_scale || c.v_scale))
    return set_last_error(FA_ERR_INVALID_ARG, "k_scale and v_scale belong to an e4m3 cache");
  const long long unit = kv_type == FA_KV_E4M3 ? 16 : 8;   // elements in 16 bytes
  const struct { const char* name; long long v; int n; } st[] = {
      {"page_stride", c.page_stride, c.num_pages}, {"slot_stride", c.slot_stride, c.page_size},
      {"head_stride", c.head_stride, c.heads_kv}};
  for (const auto& s : st) {
    if (s.n <= 1) continue;   // never multiplied by anything but 0
    if (s.v < c.head_dim)
      return set_last_error(FA_ERR_INVALID_ARG, "%s must be at least head_dim (%d elements), got %lld", s.name,
                            c.head_dim, s.v);
    if (s.v % unit)
      return set_last_error(FA_ERR_INVALID_ARG, "%s must be a multiple of 16 bytes (%lld elements), got %lld", s.name,
                            unit, s.v);
  }
  if (misaligned16(c.k) || misaligned16(c.v))
    return set_last_error(FA_ERR_INVALID_ARG, "k_cache and v_cache must be 16-byte aligned");
  if (misaligned4(c.k_scale) || misaligned4(c.v_scale))
    return set_last_error(FA_ERR_INVALID_ARG, "k_scale and v_scale must be 4-byte aligned");
  return FA_OK;
}

inline int check_row_stride(const char* name, long long stride, long long row, int rows) {
  if (rows <= 1) return FA_OK;
  if (stride < row || stride % 8)
    return set_last_error(FA_ERR_INVALID_ARG,
                          "%s must be a multiple of 8 elements and hold a whole row (%lld elements), got %lld", name,
                          row, stride);
  return FA_OK;
}

inline PagedCache make_cache(const void* k, const void* v, int kv_type, const float* k_scale, const float* v_scale,
                          long long page_stride, long long slot_stride, long long head_stride, int num_pages,
                          int page_size, int heads_kv, int head_dim) {
  PagedCache c;
  c.k = const_cast<void*>(k);
  c.v = const_cast<void*>(v);
  c.k_scale = k_scale;
  c.v_scale = v_scale;
  c.page_stride = page_stride;
  c.slot_stride = slot_stride;
  c.head_stride = head_stride;
  c.e4m3 = kv_type == FA_KV_E4M3;
  c.num_pages = num_pages;
  c.page_size = page_size;
  c.heads_kv = heads_kv;
  c.head_dim = head_dim;
  return c;
}

}  // namespace fa
