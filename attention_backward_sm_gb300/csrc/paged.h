// Launch interfaces of the paged key/value cache operators (paged.cu checks
// arguments and holds the plan and append kernels, decode.cu the attention
// of one new token).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace fa {

// A paged cache: slot s of page p, key/value head h starts at element
// p * page_stride + s * slot_stride + h * head_stride of k and of v.
struct PagedCache {
  void* k;
  void* v;
  const float* k_scale;   // [heads_kv] or nullptr (1)
  const float* v_scale;
  long long page_stride;  // elements
  long long slot_stride;
  long long head_stride;
  int e4m3;               // 1: one byte per element, else bf16
  int num_pages;
  int page_size;
  int heads_kv;
  int head_dim;
};

// n / d for 0 <= n < 2^31 by a product: with 2^shift the power of two at or
// above d and mul = ceil(2^32 (2^shift - d) / d) (+ 1 where exact), the sum
// n + floor(n mul / 2^32) over 2^shift is exact for all 32-bit n.
struct FastDiv {
  uint32_t mul;
  uint32_t shift;
  explicit FastDiv(uint32_t d = 1) : shift(0) {
    while ((1ull << shift) < d) ++shift;
    mul = static_cast<uint32_t>(((1ull << 32) * ((1ull << shift) - d)) / d + 1);
  }
  __device__ __forceinline__ int quotient(int n) const {
    return static_cast<int>((__umulhi(static_cast<uint32_t>(n), mul) + static_cast<uint32_t>(n)) >> shift);
  }
};

struct DecodeParams {
  PagedCache kv;
  const uint16_t* q;      // [batch, heads, d], rows q_row_stride elements apart
  long long q_row_stride;
  const int32_t* table;   // [batch, max_pages], rows table_stride entries apart
  long long table_stride;
  const int32_t* seq_lens;
  uint16_t* o;            // [batch, heads, d]
  float* lse;             // [batch, heads] or nullptr
  float* work;
  FastDiv page_div;       // by kv.page_size
  int max_pages;
  int batch;
  int heads;
  int window;
  float scale;
};

size_t decode_workspace_bytes(int batch, int heads, int heads_kv, int head_dim);
cudaError_t launch_decode(const DecodeParams& p, cudaStream_t s);

}  // namespace fa
