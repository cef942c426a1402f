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
  int max_pages;
  int batch;
  int heads;
  int window;
  float scale;
};

size_t decode_workspace_bytes(int batch, int heads, int heads_kv, int head_dim);
cudaError_t launch_decode(const DecodeParams& p, cudaStream_t s);

}  // namespace fa
