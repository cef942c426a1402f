// Launch interfaces of the paged key/value cache operators (paged.cu checks
// arguments and holds the plan and append kernels, decode.cu the attention
// of one new token).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>

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

// n / d for 0 <= n < 2^31 by a product, after Granlund and Montgomery
// (Division by Invariant Integers using Multiplication, 1994): with 2^shift
// the power of two at or above d and mul = floor(2^32 (2^shift - d) / d) + 1,
// the sum n + floor(n mul / 2^32) over 2^shift is exact for all 32-bit n.
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

// Programmatic dependent launch.  These kernels' launches need not wait for
// the kernel before them in the stream to be flushed; pdl_wait, before
// anything is read or written, waits until it has ended and its writes are
// visible (calls one after the other: append of 64 rows 4.1 -> 2.8 us each).
// What an earlier kernel may have written is read with plain loads: it can
// change while these kernels are already there, which ld.global.nc excludes.
// pdl_launch lets the next kernel be set up while this one still runs.  Only
// decode does that, for its combine: a decode block that was set up beside
// others found its SM's shared memory in pieces, and fewer of its neighbours
// fitted for as long as it ran (64 requests, 16 heads of 64: 97 -> 115 us
// with combine kernels that let the next decode start).
__device__ __forceinline__ void pdl_launch() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void pdl_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// Once per kernel and device: its dynamic shared memory, and the largest
// split of an SM's memory for shared memory, also for the combine kernel,
// which needs little: the split only changes on an idle SM, and that kernel's
// blocks may be the first on theirs.
inline cudaError_t prepare_once(const void* kernel, int smem, int dev, std::atomic<unsigned long long>& done) {
  cudaError_t e = cudaSuccess;
  const unsigned long long bit = dev < 64 ? (1ull << dev) : 0ull;
  if (bit && (done.load(std::memory_order_acquire) & bit)) return cudaSuccess;
  if (smem > 0) e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributePreferredSharedMemoryCarveout, cudaSharedmemCarveoutMaxShared);
  if (e == cudaSuccess && bit) done.fetch_or(bit, std::memory_order_release);
  return e;
}

template <class... Params, class... Args>
cudaError_t launch_pdl(void (*kernel)(Params...), dim3 grid, dim3 block, size_t smem, cudaStream_t s,
                       const Args&... args) {
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

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

struct Device {
  int id;
  int sms;
};

size_t decode_workspace_bytes(int batch, int heads, int heads_kv, int head_dim);
cudaError_t launch_decode(const DecodeParams& p, const Device& dev, cudaStream_t s);

}  // namespace fa
