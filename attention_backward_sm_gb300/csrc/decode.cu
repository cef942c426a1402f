// Attention of one new token per request over a paged key/value cache.
//
// For request b, query head h (key/value head h / (heads / heads_kv)) and
// the visible cached keys j in [max(0, len - window), len):
//     x_j = scale * q . k_j,  o = sum_j exp(x_j) v_j / sum_j exp(x_j),
//     lse = ln sum_j exp(x_j)
// in one pass over the keys with a running maximum and sum.  Keys whose
// block-table entry is not a page of the cache are not seen; a row that sees
// no key gets o = 0, lse = -inf.
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "paged.h"
#include "sm103.cuh"

namespace fa {
namespace {

constexpr int kWarps = 4;
constexpr float kLog2e = 1.4426950408889634f;

__device__ __forceinline__ float2 e4m3_pair(uint32_t two) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(static_cast<uint16_t>(two)));
  return __half22float2(*reinterpret_cast<__half2*>(&h));
}

// D / 32 consecutive elements of a cache row, as floats.
template <int N, bool E4M3>
__device__ __forceinline__ void load_row(const void* base, long long at, float (&x)[N]) {
#pragma unroll
  for (int i = 0; i < N; i += 2) {
    if constexpr (E4M3) {
      const float2 f = e4m3_pair(*reinterpret_cast<const uint16_t*>(static_cast<const uint8_t*>(base) + at + i));
      x[i] = f.x;
      x[i + 1] = f.y;
    } else {
      const uint32_t u = *reinterpret_cast<const uint32_t*>(static_cast<const uint16_t*>(base) + at + i);
      x[i] = __uint_as_float(u << 16);
      x[i + 1] = __uint_as_float(u & 0xFFFF0000u);
    }
  }
}

// One block per (request, query head); warp w takes keys w, w + kWarps, ...
// and the warps' softmax states are joined at the end.
template <int D, bool E4M3>
__global__ void __launch_bounds__(kWarps * 32) decode_kernel(const DecodeParams p) {
  constexpr int N = D / 32;
  __shared__ float s_m[kWarps], s_l[kWarps], s_o[kWarps][D];
  const int b = blockIdx.x / p.heads, h = blockIdx.x % p.heads;
  const int hk = h / (p.heads / p.kv.heads_kv);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int len = min(max(p.seq_lens[b], 0), p.max_pages * p.kv.page_size);
  const int first = p.window > 0 ? max(0, len - p.window) : 0;
  const float ks = p.kv.k_scale ? p.kv.k_scale[hk] : 1.f, vs = p.kv.v_scale ? p.kv.v_scale[hk] : 1.f;
  float q[N], o[N], m = -INFINITY, l = 0.f;
  load_row<N, false>(p.q, b * p.q_row_stride + static_cast<long long>(h) * D + lane * N, q);
#pragma unroll
  for (int i = 0; i < N; ++i) o[i] = 0.f;
  for (int j = first + warp; j < len; j += kWarps) {
    const int page = p.table[b * p.table_stride + j / p.kv.page_size];
    if (page < 0 || page >= p.kv.num_pages) continue;
    const long long at = page * p.kv.page_stride + (j % p.kv.page_size) * p.kv.slot_stride + hk * p.kv.head_stride +
                         lane * N;
    float k[N], v[N];
    load_row<N, E4M3>(p.kv.k, at, k);
    load_row<N, E4M3>(p.kv.v, at, v);
    float x = 0.f;
#pragma unroll
    for (int i = 0; i < N; ++i) x = fmaf(q[i], k[i], x);
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) x += __shfl_xor_sync(0xffffffffu, x, off);
    x *= p.scale * ks * kLog2e;
    const float top = fmaxf(m, x);
    const float keep = exp2f(m - top), e = exp2f(x - top);
    m = top;
    l = l * keep + e;
#pragma unroll
    for (int i = 0; i < N; ++i) o[i] = fmaf(o[i], keep, e * v[i]);
  }
  if (lane == 0) {
    s_m[warp] = m;
    s_l[warp] = l;
  }
#pragma unroll
  for (int i = 0; i < N; ++i) s_o[warp][lane * N + i] = o[i];
  __syncthreads();
  float top = -INFINITY;
  for (int w = 0; w < kWarps; ++w) top = fmaxf(top, s_m[w]);
  float total = 0.f;
  for (int w = 0; w < kWarps; ++w)
    if (s_l[w] != 0.f) total += s_l[w] * exp2f(s_m[w] - top);
  const long long row = static_cast<long long>(b) * p.heads + h;
  for (int c = threadIdx.x; c < D; c += kWarps * 32) {
    float sum = 0.f;
    for (int w = 0; w < kWarps; ++w)
      if (s_l[w] != 0.f) sum += s_o[w][c] * exp2f(s_m[w] - top);
    const float out = total == 0.f ? 0.f : sum / total * vs;
    p.o[row * D + c] = static_cast<uint16_t>(pack_bf16x2(out, out) & 0xffffu);
  }
  if (p.lse && threadIdx.x == 0) p.lse[row] = total == 0.f ? -INFINITY : (top + log2f(total)) * 0.6931471805599453f;
}

template <int D>
cudaError_t launch_d(const DecodeParams& p, cudaStream_t s) {
  const int grid = p.batch * p.heads;
  if (p.kv.e4m3) decode_kernel<D, true><<<grid, kWarps * 32, 0, s>>>(p);
  else decode_kernel<D, false><<<grid, kWarps * 32, 0, s>>>(p);
  return cudaGetLastError();
}

}  // namespace

size_t decode_workspace_bytes(int, int, int, int) { return 0; }

cudaError_t launch_decode(const DecodeParams& p, cudaStream_t s) {
  if (p.kv.head_dim == 64) return launch_d<64>(p, s);
  if (p.kv.head_dim == 128) return launch_d<128>(p, s);
  return launch_d<256>(p, s);
}

}  // namespace fa
