// Rotation of queries and keys by their positions, with an optional norm of
// every head: C entry points and kernels (forward, gradient, and forward
// straight into the paged cache).
//
// A head x of d values at position p:
//     n   = x / sqrt(mean(x^2) + eps) * w           (n = x without a weight)
//     y_a = mscale (n_a cos t - n_b sin t),  y_b = mscale (n_b cos t + n_a sin t)
// for the pairs i of the first `rotary` values, (a, b) = (2i, 2i + 1) or
// (i, i + rotary / 2), t = p * theta_i; the values past them stay n.  Its
// gradient turns dy back, g = mscale R(-t) dy, and with a norm
//     u  = x / sqrt(mean(x^2) + eps),   dw = sum over rows of g u,
//     dx = (g w - u mean(g w u)) / sqrt(mean(x^2) + eps).
//
// Angles.  theta_i comes as a 64-bit fixed-point fraction of a turn, so
// p * theta_i mod 2^64 is the angle of any 32-bit position without the loss of
// a 32-bit product (at position 131072 that would be 0.008 radians).  The upper
// 32 bits of it, as fp32, go to sincospif.
//
// All of it is one pass over the rows, bound by HBM: a thread holds 16 values
// of a head (two pieces of 16 bytes that belong together under the rotation),
// d / 16 threads make a head, and the sines and cosines of a block's tokens are
// worked out once, in shared memory, for all of their heads.  Everything
// between the loads and the one rounding at the end is fp32.
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>
#include <stdio.h>

#include <atomic>
#include <type_traits>

#include "../../include/fabwd.h"
#include "checks.h"
#include "internal.h"
#include "paged.h"
#include "quantise.cuh"
#include "sm103.cuh"

namespace {

using namespace fa;

constexpr int kThreads = 256;
constexpr int kMostTokens = 8;       // of a block at a time
constexpr int kReduceThreads = 256;
constexpr int kBwdBlocksPerSm = 3;   // blocks that walk through the tokens, each leaves one partial sum of the weights' gradients
constexpr int kMostSms = 152;

struct Rows {
  const uint16_t* in;    // [tokens, heads, d], rows in_stride elements apart
  const uint16_t* x;     // gradient: the forward's input
  uint16_t* out;
  long long in_stride;
  long long x_stride;
  long long out_stride;
  const void* weight;    // [d] or nullptr: no norm
};

struct RopeParams {
  Rows q, k;
  const uint16_t* v;     // with a cache
  long long v_stride;
  const int32_t* positions;
  const unsigned long long* freqs;   // [rotary / 2] turns * 2^64
  float* partial;        // gradient: [blocks][2][d]
  PagedCache kv;
  const int64_t* slots;
  FastDiv page_div;
  FastDiv head_div;      // by the heads of a token, of all kinds
  int rotary;
  int half;              // pairs (i, i + rotary / 2), else (2i, 2i + 1)
  int weight_f32;
  float mscale;
  float sin_scale;       // mscale, or -mscale to turn back
  float eps;
  int num_tokens;
  int tokens_per_block;
  int heads;
  int heads_kv;
};

// cos and sin of a block's tokens: [2][tokens][rotary / 2].
__device__ __forceinline__ void fill_turns(const RopeParams& p, long long t0, int tokens, float* turns) {
  const int pairs = p.rotary / 2, total = tokens * pairs;
  float* const sines = turns + p.tokens_per_block * pairs;
  for (int i = threadIdx.x; i < total; i += kThreads) {
    const int t = i / pairs;
    const unsigned long long phase =
        static_cast<unsigned long long>(static_cast<long long>(p.positions[t0 + t])) * p.freqs[i - t * pairs];
    float s, c;
    sincospif(static_cast<float>(static_cast<int>(phase >> 32)) * 0x1p-31f, &s, &c);
    turns[i] = c * p.mscale;
    sines[i] = s * p.sin_scale;
  }
}

__device__ __forceinline__ float weight_at(const void* w, int f32, int i) {
  return f32 ? static_cast<const float*>(w)[i]
             : __uint_as_float(static_cast<uint32_t>(static_cast<const uint16_t*>(w)[i]) << 16);
}

// A thread's place in a head: its two pieces of 8 values and its 8 pairs.
struct Place {
  int a, b;       // first elements of the pieces
  bool turned;
  __device__ __forceinline__ Place(const RopeParams& p, int u) {
    turned = u < p.rotary / 16;
    if (!p.half) {
      a = 16 * u;
      b = a + 8;
    } else if (turned) {
      a = 8 * u;
      b = a + p.rotary / 2;
    } else {
      a = 16 * u;   // rotary + 16 (u - rotary / 16)
      b = a + 8;
    }
  }
};

__device__ __forceinline__ void unpack8(const uint4& v, float* x) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = bf_lo(w[i]);
    x[2 * i + 1] = bf_hi(w[i]);
  }
}
__device__ __forceinline__ uint4 pack8(const float* x) {
  return make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]),
                    pack_bf16x2(x[6], x[7]));
}
__device__ __forceinline__ void load8(const float* from, float* x) {
  const float4 a = *reinterpret_cast<const float4*>(from), b = *reinterpret_cast<const float4*>(from + 4);
  x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w;
  x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
}

// x[0..7] is piece a, x[8..15] piece b; c and s of the thread's 8 pairs.
__device__ __forceinline__ void turn16(float* x, const float* c, const float* s, bool half) {
  if (half) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float a = x[i], b = x[8 + i];
      x[i] = a * c[i] - b * s[i];
      x[8 + i] = b * c[i] + a * s[i];
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float a = x[2 * i], b = x[2 * i + 1];
      x[2 * i] = a * c[i] - b * s[i];
      x[2 * i + 1] = b * c[i] + a * s[i];
    }
  }
}

// Sum over the D / 16 threads of a head.
template <int D>
__device__ __forceinline__ float head_sum(float v) {
#pragma unroll
  for (int off = D / 32; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
  return v;
}

__device__ __forceinline__ uint4 load16(const uint16_t* p) { return ldg_stream(p); }

// ---------------------------------------------------------------- forward
template <int D, bool NORM, bool CACHE>
__global__ void __launch_bounds__(kThreads) rope_kernel(const RopeParams p) {
  constexpr int TPH = D / 16, SLOTS = kThreads / TPH;
  extern __shared__ __align__(16) float turns[];
  __shared__ __align__(16) float weights[NORM ? 2 * D : 4];
  const int u = threadIdx.x % TPH, slot = threadIdx.x / TPH;
  const Place at(p, u);
  const int per_token = p.heads + (CACHE ? 2 : 1) * p.heads_kv;
  const long long t0 = static_cast<long long>(blockIdx.x) * p.tokens_per_block;
  const int tokens = static_cast<int>(min(static_cast<long long>(p.tokens_per_block), p.num_tokens - t0));
  const int items = tokens * per_token;
  pdl_wait();

  struct Item {
    uint4 a, b;
    int t, h;
  };
  auto load = [&](int n, Item& it) {
    it.t = -1;
    it.a = it.b = make_uint4(0, 0, 0, 0);
    if (n >= items) return;
    it.t = p.head_div.quotient(n);
    it.h = n - it.t * per_token;
    const long long t = t0 + it.t;
    const uint16_t* from;
    if (it.h < p.heads) from = p.q.in + t * p.q.in_stride + it.h * D;
    else if (!CACHE || it.h < p.heads + p.heads_kv) from = p.k.in + t * p.k.in_stride + (it.h - p.heads) * D;
    else from = p.v + t * p.v_stride + (it.h - p.heads - p.heads_kv) * D;
    it.a = load16(from + at.a);
    it.b = load16(from + at.b);
  };
  Item next;
  load(slot, next);   // on its way while the sines are worked out
  if constexpr (NORM) {
    for (int i = threadIdx.x; i < 2 * D; i += kThreads) {
      const void* const w = i < D ? p.q.weight : p.k.weight;
      weights[i] = w ? weight_at(w, p.weight_f32, i % D) : 1.f;
    }
  }
  fill_turns(p, t0, tokens, turns);
  __syncthreads();

  const int pairs = p.rotary / 2;
  for (int n0 = 0; n0 < items; n0 += SLOTS) {
    const Item it = next;
    load(n0 + SLOTS + slot, next);
    const bool is_q = it.h < p.heads, is_v = CACHE && it.h >= p.heads + p.heads_kv;
    float x[16];
    unpack8(it.a, x);
    unpack8(it.b, x + 8);
    if constexpr (NORM) {
      float sum = 0.f;
#pragma unroll
      for (int i = 0; i < 16; ++i) sum = fmaf(x[i], x[i], sum);
      sum = head_sum<D>(sum);
      if (!is_v && (is_q ? p.q.weight : p.k.weight) != nullptr) {
        const float inv = rsqrtf(fmaf(sum, 1.f / D, p.eps));
        float w[16];
        load8(weights + (is_q ? 0 : D) + at.a, w);
        load8(weights + (is_q ? 0 : D) + at.b, w + 8);
#pragma unroll
        for (int i = 0; i < 16; ++i) x[i] *= inv * w[i];
      }
    }
    if (it.t < 0) continue;
    if (at.turned && !is_v) {
      float c[8], s[8];
      const float* const from = turns + it.t * pairs + 8 * u;
      load8(from, c);
      load8(from + p.tokens_per_block * pairs, s);
      turn16(x, c, s, p.half);
    }
    const long long t = t0 + it.t;
    if (!CACHE || is_q) {
      uint16_t* const to = is_q ? p.q.out + t * p.q.out_stride + it.h * D
                                : p.k.out + t * p.k.out_stride + (it.h - p.heads) * D;
      *reinterpret_cast<uint4*>(to + at.a) = pack8(x);
      *reinterpret_cast<uint4*>(to + at.b) = pack8(x + 8);
    } else {
      const long long s = p.slots[t], num_slots = static_cast<long long>(p.kv.num_pages) * p.kv.page_size;
      if (s < 0 || s >= num_slots) continue;
      const long long page = s <= 0x7fffffffll ? p.page_div.quotient(static_cast<int>(s)) : s / p.kv.page_size;
      const int h = it.h - p.heads - (is_v ? p.heads_kv : 0);
      const long long e = page * p.kv.page_stride + (s - page * p.kv.page_size) * p.kv.slot_stride + h * p.kv.head_stride;
      void* const cache = is_v ? p.kv.v : p.kv.k;
      if (p.kv.e4m3) {
        uint8_t* const to = static_cast<uint8_t*>(cache) + e;
        const float* const scales = is_v ? p.kv.v_scale : p.kv.k_scale;
        uint2 a, b;
        if (is_v) {   // as fa_kv_append stores them
          const Scale sc(scales, h);
          a = quantise8(it.a, sc);
          b = quantise8(it.b, sc);
        } else {
          // rounded once: the turned values do not pass through bf16
          const float sc = scales ? scales[h] : 1.f;
#pragma unroll
          for (int i = 0; i < 16; ++i) x[i] = __fdiv_rn(x[i], sc);
          a = make_uint2(e4m3x2(x[0], x[1]) | e4m3x2(x[2], x[3]) << 16, e4m3x2(x[4], x[5]) | e4m3x2(x[6], x[7]) << 16);
          b = make_uint2(e4m3x2(x[8], x[9]) | e4m3x2(x[10], x[11]) << 16,
                         e4m3x2(x[12], x[13]) | e4m3x2(x[14], x[15]) << 16);
        }
        *reinterpret_cast<uint2*>(to + at.a) = a;
        *reinterpret_cast<uint2*>(to + at.b) = b;
      } else {
        uint16_t* const to = static_cast<uint16_t*>(cache) + e;
        *reinterpret_cast<uint4*>(to + at.a) = is_v ? it.a : pack8(x);
        *reinterpret_cast<uint4*>(to + at.b) = is_v ? it.b : pack8(x + 8);
      }
    }
  }
}

// ---------------------------------------------------------------- gradient
// Blocks walk through the tokens, the query heads of all of theirs first, then
// the key heads, so that one set of 16 sums per thread is enough for the
// weights' gradients.  Each block leaves one partial sum per weight;
// weight_kernel adds them in a fixed order.
template <int D>
__global__ void __launch_bounds__(kThreads, kBwdBlocksPerSm) rope_bwd_kernel(const RopeParams p) {
  constexpr int TPH = D / 16, SLOTS = kThreads / TPH, WARPS = kThreads / 32;
  extern __shared__ __align__(16) float turns[];
  __shared__ __align__(16) float weights[D];
  __shared__ __align__(16) float sums[WARPS][D];
  const int u = threadIdx.x % TPH, slot = threadIdx.x / TPH, warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const Place at(p, u);
  const int pairs = p.rotary / 2;
  pdl_wait();
  pdl_launch();
  for (int tensor = 0; tensor < 2; ++tensor) {
    const Rows& r = tensor ? p.k : p.q;
    const int heads = tensor ? p.heads_kv : p.heads;
    const bool norm = r.weight != nullptr;
    float acc[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) acc[i] = 0.f;
    __syncthreads();
    if (norm)
      for (int i = threadIdx.x; i < D; i += kThreads) weights[i] = weight_at(r.weight, p.weight_f32, i);
    for (long long t0 = static_cast<long long>(blockIdx.x) * p.tokens_per_block; heads > 0 && t0 < p.num_tokens;
         t0 += static_cast<long long>(gridDim.x) * p.tokens_per_block) {
      const int tokens = static_cast<int>(min(static_cast<long long>(p.tokens_per_block), p.num_tokens - t0));
      const int items = tokens * heads;
      struct Item {
        uint4 ga, gb, xa, xb;
        int t, h;
      };
      auto load = [&](int n, Item& it) {
        it.t = -1;
        it.ga = it.gb = it.xa = it.xb = make_uint4(0, 0, 0, 0);
        if (n >= items) return;
        it.t = n / heads;
        it.h = n - it.t * heads;
        const uint16_t* const g = r.in + (t0 + it.t) * r.in_stride + it.h * D;
        it.ga = load16(g + at.a);
        it.gb = load16(g + at.b);
        if (norm) {
          const uint16_t* const x = r.x + (t0 + it.t) * r.x_stride + it.h * D;
          it.xa = load16(x + at.a);
          it.xb = load16(x + at.b);
        }
      };
      Item next;
      load(slot, next);
      __syncthreads();   // the tokens before are done with their turns
      fill_turns(p, t0, tokens, turns);
      __syncthreads();
      for (int n0 = 0; n0 < items; n0 += SLOTS) {
        const Item it = next;
        load(n0 + SLOTS + slot, next);
        float g[16], x[16];
        unpack8(it.ga, g);
        unpack8(it.gb, g + 8);
        if (at.turned && it.t >= 0) {
          float c[8], s[8];
          const float* const from = turns + it.t * pairs + 8 * u;
          load8(from, c);
          load8(from + p.tokens_per_block * pairs, s);
          turn16(g, c, s, p.half);
        }
        if (norm) {
          unpack8(it.xa, x);
          unpack8(it.xb, x + 8);
          float sum = 0.f;
#pragma unroll
          for (int i = 0; i < 16; ++i) sum = fmaf(x[i], x[i], sum);
          const float inv = rsqrtf(fmaf(head_sum<D>(sum), 1.f / D, p.eps));
          float w[16], along = 0.f;
          load8(weights + at.a, w);
          load8(weights + at.b, w + 8);
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            x[i] *= inv;
            if (it.t >= 0) acc[i] = fmaf(g[i], x[i], acc[i]);
            g[i] *= w[i];
            along = fmaf(g[i], x[i], along);
          }
          along = head_sum<D>(along) * (1.f / D);
#pragma unroll
          for (int i = 0; i < 16; ++i) g[i] = inv * fmaf(-x[i], along, g[i]);
        }
        if (it.t < 0) continue;
        uint16_t* const to = r.out + (t0 + it.t) * r.out_stride + it.h * D;
        *reinterpret_cast<uint4*>(to + at.a) = pack8(g);
        *reinterpret_cast<uint4*>(to + at.b) = pack8(g + 8);
      }
    }
    if (norm) {
      // the heads of a warp, then the warps, in order
#pragma unroll
      for (int i = 0; i < 16; ++i)
#pragma unroll
        for (int off = TPH; off < 32; off <<= 1) acc[i] += __shfl_xor_sync(0xffffffffu, acc[i], off);
      if (lane < TPH) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          sums[warp][at.a + i] = acc[i];
          sums[warp][at.b + i] = acc[8 + i];
        }
      }
      __syncthreads();
      for (int i = threadIdx.x; i < D; i += kThreads) {
        float sum = 0.f;
#pragma unroll
        for (int w = 0; w < WARPS; ++w) sum += sums[w][i];
        p.partial[(static_cast<long long>(blockIdx.x) * 2 + tensor) * D + i] = sum;
      }
    }
  }
}

// dw[i] = the sum of the blocks' partial sums: 8 columns per block, 32 threads
// each.
template <int D>
__global__ void __launch_bounds__(kReduceThreads) weight_kernel(const float* partial, int blocks, float* dq_weight,
                                                                float* dk_weight) {
  __shared__ float part[kReduceThreads / 8][8];
  const int c = threadIdx.x % 8, r = threadIdx.x / 8, column = blockIdx.x * 8 + c;   // of [2][D]
  pdl_wait();
  float sum = 0.f;
  for (int b = r; b < blocks; b += kReduceThreads / 8) sum += partial[static_cast<long long>(b) * 2 * D + column];
  part[r][c] = sum;
  __syncthreads();
  if (r > 0) return;
  for (int i = 1; i < kReduceThreads / 8; ++i) sum += part[i][c];
  float* const to = column < D ? dq_weight : dk_weight;
  if (to) to[column % D] = sum;
}

// ---------------------------------------------------------------- host
template <class F>
auto with_dim(int d, F f) {
  using std::integral_constant;
  if (d == 64) return f(integral_constant<int, 64>());
  if (d == 128) return f(integral_constant<int, 128>());
  return f(integral_constant<int, 256>());
}

// Whether rows [n, row] of two arrays may have elements in common.
bool clash(const void* a, long long a_stride, long long a_row, const void* b, long long b_stride, long long b_row,
           long long n) {
  if (n == 0 || a_row == 0 || b_row == 0) return false;
  const uintptr_t a0 = reinterpret_cast<uintptr_t>(a), b0 = reinterpret_cast<uintptr_t>(b);
  const uintptr_t a1 = a0 + 2ull * ((n - 1) * a_stride + a_row), b1 = b0 + 2ull * ((n - 1) * b_stride + b_row);
  if (a1 <= b0 || b1 <= a0) return false;
  if (a_stride != b_stride || n == 1) return true;
  // rows of one larger array: where b's rows start in a's
  const unsigned long long s = 2ull * a_stride;
  const unsigned long long d = b0 >= a0 ? (b0 - a0) % s : (s - (a0 - b0) % s) % s;
  return d < 2ull * a_row || d + 2ull * b_row > s;
}

struct Array {
  const char* name;
  const void* p;
  long long stride;
  long long row;
  bool out;
};

// Row strides, alignment, NULL, and that outputs overlap nothing (but what they
// take the place of: arrays i and i + 1 may be one where `pair` says so).
int check_rows(const Array* a, int n, long long tokens, unsigned pairs) {
  int rc;
  for (int i = 0; i < n; ++i) {
    if (a[i].row == 0) continue;
    char stride[40];
    snprintf(stride, sizeof(stride), "%s_row_stride", a[i].name);
    if ((rc = check_row_stride(stride, a[i].stride, a[i].row, static_cast<int>(tokens)))) return rc;
    if (tokens > 0 && !a[i].p) return set_last_error(FA_ERR_INVALID_ARG, "%s is NULL", a[i].name);
    if (misaligned16(a[i].p)) return set_last_error(FA_ERR_INVALID_ARG, "%s must be 16-byte aligned", a[i].name);
  }
  for (int i = 0; i < n; ++i)
    for (int j = 0; j < n; ++j) {
      if (i == j || !a[i].out || (a[j].out && j < i)) continue;
      const bool same = a[i].p == a[j].p && (tokens <= 1 || a[i].stride == a[j].stride) && a[i].row == a[j].row;
      if (same && j + 1 == i && (pairs >> j & 1)) continue;
      if (clash(a[i].p, a[i].stride, a[i].row, a[j].p, a[j].stride, a[j].row, tokens))
        return set_last_error(FA_ERR_INVALID_ARG, "%s must not overlap %s", a[i].name, a[j].name);
    }
  return FA_OK;
}

int check_common(const RopeParams& p, int head_dim, int layout, int weight_type) {
  if (head_dim != 64 && head_dim != 128 && head_dim != 256)
    return set_last_error(FA_ERR_UNSUPPORTED, "head_dim must be 64, 128 or 256, got %d", head_dim);
  if (p.num_tokens < 0) return set_last_error(FA_ERR_INVALID_ARG, "num_tokens must be >= 0, got %d", p.num_tokens);
  if (p.heads < 0 || p.heads_kv < 0)
    return set_last_error(FA_ERR_INVALID_ARG, "heads and heads_kv must be >= 0, got %d and %d", p.heads, p.heads_kv);
  if (static_cast<long long>(p.heads) * head_dim > 65535 * 64 || static_cast<long long>(p.heads_kv) * head_dim > 65535 * 64)
    return set_last_error(FA_ERR_UNSUPPORTED, "heads * head_dim too large (%d and %d of %d)", p.heads, p.heads_kv,
                          head_dim);
  if (p.rotary < 0 || p.rotary > head_dim || p.rotary % 16 != 0)
    return set_last_error(FA_ERR_UNSUPPORTED, "rotary_dim must be a multiple of 16 from 0 to head_dim (%d), got %d",
                          head_dim, p.rotary);
  if (layout != FA_ROPE_HALF && layout != FA_ROPE_INTERLEAVED)
    return set_last_error(FA_ERR_INVALID_ARG, "layout must be 0 (half) or 1 (interleaved), got %d", layout);
  if (weight_type != FA_WEIGHT_BF16 && weight_type != FA_WEIGHT_F32)
    return set_last_error(FA_ERR_INVALID_ARG, "weight_type must be 0 (bf16) or 1 (float32), got %d", weight_type);
  if (!isfinite(p.mscale)) return set_last_error(FA_ERR_INVALID_ARG, "mscale must be finite");
  if (!(p.eps >= 0.f) || !isfinite(p.eps)) return set_last_error(FA_ERR_INVALID_ARG, "eps must be finite and >= 0");
  if (p.rotary > 0 && p.num_tokens > 0 && (!p.positions || !p.freqs))
    return set_last_error(FA_ERR_INVALID_ARG, "positions or freqs is NULL");
  if (misaligned4(p.positions) || (reinterpret_cast<uintptr_t>(p.freqs) & 7u))
    return set_last_error(FA_ERR_INVALID_ARG, "positions must be 4-byte aligned, freqs 8-byte");
  const uintptr_t unit = weight_type == FA_WEIGHT_F32 ? 3u : 1u;
  if ((reinterpret_cast<uintptr_t>(p.q.weight) | reinterpret_cast<uintptr_t>(p.k.weight)) & unit)
    return set_last_error(FA_ERR_INVALID_ARG, "q_weight and k_weight must be aligned to their type");
  return FA_OK;
}

RopeParams make_params(const void* positions, const void* freqs, int rotary, int layout, float mscale, bool back,
                       const void* q_weight, const void* k_weight, int weight_type, float eps, int tokens, int heads,
                       int heads_kv) {
  RopeParams p = RopeParams();
  p.positions = static_cast<const int32_t*>(positions);
  p.freqs = static_cast<const unsigned long long*>(freqs);
  p.rotary = rotary;
  p.half = layout == FA_ROPE_HALF;
  p.mscale = mscale;
  p.sin_scale = back ? -mscale : mscale;
  p.q.weight = q_weight;
  p.k.weight = k_weight;
  p.weight_f32 = weight_type == FA_WEIGHT_F32;
  p.eps = eps;
  p.num_tokens = tokens;
  p.heads = heads;
  p.heads_kv = heads_kv;
  return p;
}

cudaError_t launch_forward(RopeParams& p, int head_dim, bool cache, const Device& dev, cudaStream_t s) {
  const int per_token = p.heads + (cache ? 2 : 1) * p.heads_kv;
  // One token per block until every SM has four blocks.
  const int per = p.num_tokens / (4 * dev.sms);
  p.tokens_per_block = per < 1 ? 1 : per > kMostTokens ? kMostTokens : per;
  p.head_div = FastDiv(static_cast<uint32_t>(per_token));
  const int grid = (p.num_tokens + p.tokens_per_block - 1) / p.tokens_per_block;
  const size_t smem = static_cast<size_t>(p.tokens_per_block) * p.rotary * sizeof(float);
  const bool norm = p.q.weight || p.k.weight;
  return with_dim(head_dim, [&](auto d) {
    constexpr int D = decltype(d)::value;
    auto* const kernel = cache ? (norm ? rope_kernel<D, true, true> : rope_kernel<D, false, true>)
                               : (norm ? rope_kernel<D, true, false> : rope_kernel<D, false, false>);
    return launch_pdl(kernel, dim3(grid), dim3(kThreads), smem, s, p);
  });
}

}  // namespace

extern "C" {

int fa_qk_rope(const fa_bf16* q, const fa_bf16* k, long long q_row_stride, long long k_row_stride,
               const int32_t* positions, const uint64_t* freqs, int rotary_dim, int layout, float mscale,
               const void* q_weight, const void* k_weight, int weight_type, float eps, int num_tokens, int heads,
               int heads_kv, int head_dim, fa_bf16* q_out, fa_bf16* k_out, long long q_out_row_stride,
               long long k_out_row_stride, fa_stream_t stream) {
  RopeParams p = make_params(positions, freqs, rotary_dim, layout, mscale, false, q_weight, k_weight, weight_type, eps,
                             num_tokens, heads, heads_kv);
  int rc = check_common(p, head_dim, layout, weight_type);
  if (rc) return rc;
  const long long wq = static_cast<long long>(heads) * head_dim, wk = static_cast<long long>(heads_kv) * head_dim;
  const Array arrays[] = {{"q", q, q_row_stride, wq, false}, {"q_out", q_out, q_out_row_stride, wq, true},
                          {"k", k, k_row_stride, wk, false}, {"k_out", k_out, k_out_row_stride, wk, true}};
  if ((rc = check_rows(arrays, 4, num_tokens, 0x5))) return rc;
  if (num_tokens == 0 || heads + heads_kv == 0) return ok();
  Device dev;
  if ((rc = check_device(dev))) return rc;
  p.q.in = q, p.q.in_stride = q_row_stride, p.q.out = q_out, p.q.out_stride = q_out_row_stride;
  p.k.in = k, p.k.in_stride = k_row_stride, p.k.out = k_out, p.k.out_stride = k_out_row_stride;
  cudaError_t e = launch_forward(p, head_dim, false, dev, reinterpret_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "rope launch");
  return ok();
}

int fa_qk_rope_append(const fa_bf16* q, const fa_bf16* k, const fa_bf16* v, long long q_row_stride,
                      long long k_row_stride, long long v_row_stride, const int32_t* positions, const uint64_t* freqs,
                      int rotary_dim, int layout, float mscale, const void* q_weight, const void* k_weight,
                      int weight_type, float eps, int num_tokens, int heads, fa_bf16* q_out,
                      long long q_out_row_stride, const int64_t* slots, void* k_cache, void* v_cache, int kv_type,
                      const float* k_scale, const float* v_scale, long long page_stride, long long slot_stride,
                      long long head_stride, int num_pages, int page_size, int heads_kv, int head_dim,
                      fa_stream_t stream) {
  RopeParams p = make_params(positions, freqs, rotary_dim, layout, mscale, false, q_weight, k_weight, weight_type, eps,
                             num_tokens, heads, heads_kv);
  p.kv = make_cache(k_cache, v_cache, kv_type, k_scale, v_scale, page_stride, slot_stride, head_stride, num_pages,
                    page_size, heads_kv, head_dim);
  int rc = check_cache(p.kv, kv_type);
  if (rc) return rc;
  if ((rc = check_common(p, head_dim, layout, weight_type))) return rc;
  const long long wq = static_cast<long long>(heads) * head_dim, wk = static_cast<long long>(heads_kv) * head_dim;
  const Array arrays[] = {{"q", q, q_row_stride, wq, false}, {"q_out", q_out, q_out_row_stride, wq, true},
                          {"k", k, k_row_stride, wk, false}, {"v", v, v_row_stride, wk, false}};
  if ((rc = check_rows(arrays, 4, num_tokens, 0x1))) return rc;
  if (num_tokens == 0) return ok();
  if (!slots || (num_pages > 0 && (!k_cache || !v_cache)))
    return set_last_error(FA_ERR_INVALID_ARG, "a device pointer is NULL");
  if (reinterpret_cast<uintptr_t>(slots) & 7u)
    return set_last_error(FA_ERR_INVALID_ARG, "slots must be 8-byte aligned");
  Device dev;
  if ((rc = check_device(dev))) return rc;
  p.q.in = q, p.q.in_stride = q_row_stride, p.q.out = q_out, p.q.out_stride = q_out_row_stride;
  p.k.in = k, p.k.in_stride = k_row_stride;
  p.v = v, p.v_stride = v_row_stride;
  p.slots = slots;
  p.page_div = FastDiv(static_cast<uint32_t>(page_size));
  cudaError_t e = launch_forward(p, head_dim, true, dev, reinterpret_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "rope append launch");
  return ok();
}

size_t fa_qk_rope_bwd_workspace_size(int head_dim) {
  if (head_dim != 64 && head_dim != 128 && head_dim != 256) {
    set_last_error(FA_ERR_UNSUPPORTED, "head_dim must be 64, 128 or 256, got %d", head_dim);
    return 0;
  }
  ok();
  return static_cast<size_t>(kMostSms) * kBwdBlocksPerSm * 2 * head_dim * sizeof(float);
}

int fa_qk_rope_bwd(const fa_bf16* dq_out, const fa_bf16* dk_out, long long dq_out_row_stride,
                   long long dk_out_row_stride, const fa_bf16* q, const fa_bf16* k, long long q_row_stride,
                   long long k_row_stride, const int32_t* positions, const uint64_t* freqs, int rotary_dim, int layout,
                   float mscale, const void* q_weight, const void* k_weight, int weight_type, float eps,
                   int num_tokens, int heads, int heads_kv, int head_dim, fa_bf16* dq, fa_bf16* dk,
                   long long dq_row_stride, long long dk_row_stride, float* dq_weight, float* dk_weight,
                   void* workspace, size_t workspace_bytes, fa_stream_t stream) {
  RopeParams p = make_params(positions, freqs, rotary_dim, layout, mscale, true, q_weight, k_weight, weight_type, eps,
                             num_tokens, heads, heads_kv);
  int rc = check_common(p, head_dim, layout, weight_type);
  if (rc) return rc;
  const long long wq = static_cast<long long>(heads) * head_dim, wk = static_cast<long long>(heads_kv) * head_dim;
  const Array arrays[] = {{"dq_out", dq_out, dq_out_row_stride, wq, false}, {"dq", dq, dq_row_stride, wq, true},
                          {"dk_out", dk_out, dk_out_row_stride, wk, false}, {"dk", dk, dk_row_stride, wk, true},
                          {"q", q, q_row_stride, q_weight ? wq : 0, false},
                          {"k", k, k_row_stride, k_weight ? wk : 0, false}};
  if ((rc = check_rows(arrays, 6, num_tokens, 0x5))) return rc;
  if ((q_weight && !dq_weight) || (k_weight && !dk_weight))
    return set_last_error(FA_ERR_INVALID_ARG, "a weight's gradient is NULL");
  if (misaligned4(dq_weight) || misaligned4(dk_weight))
    return set_last_error(FA_ERR_INVALID_ARG, "dq_weight and dk_weight must be 4-byte aligned");
  const bool norm = q_weight || k_weight;
  const size_t need = fa_qk_rope_bwd_workspace_size(head_dim);
  if (norm && (!workspace || workspace_bytes < need))
    return set_last_error(FA_ERR_INVALID_ARG, "workspace of %zu bytes needed, got %zu", need, workspace_bytes);
  if (misaligned16(workspace)) return set_last_error(FA_ERR_INVALID_ARG, "workspace must be 16-byte aligned");
  if (!norm && (num_tokens == 0 || heads + heads_kv == 0)) return ok();
  Device dev;
  if ((rc = check_device(dev))) return rc;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  p.q.in = dq_out, p.q.in_stride = dq_out_row_stride, p.q.out = dq, p.q.out_stride = dq_row_stride;
  p.k.in = dk_out, p.k.in_stride = dk_out_row_stride, p.k.out = dk, p.k.out_stride = dk_row_stride;
  if (!norm) {
    cudaError_t e = launch_forward(p, head_dim, false, dev, s);
    if (e != cudaSuccess) return cuda_fail(e, "rope gradient launch");
    return ok();
  }
  p.q.x = q, p.q.x_stride = q_row_stride;
  p.k.x = k, p.k.x_stride = k_row_stride;
  p.partial = static_cast<float*>(workspace);
  const int most = kBwdBlocksPerSm * (dev.sms < kMostSms ? dev.sms : kMostSms);
  const int per = num_tokens / most;
  p.tokens_per_block = per < 1 ? 1 : per > kMostTokens ? kMostTokens : per;
  const int chunks = (num_tokens + p.tokens_per_block - 1) / p.tokens_per_block;
  const int blocks = chunks < 1 ? 1 : chunks < most ? chunks : most;   // without tokens the weights' gradients are 0
  const size_t smem = static_cast<size_t>(p.tokens_per_block) * rotary_dim * sizeof(float);
  cudaError_t e = with_dim(head_dim, [&](auto d) {
    constexpr int D = decltype(d)::value;
    cudaError_t e = launch_pdl(rope_bwd_kernel<D>, dim3(blocks), dim3(kThreads), smem, s, p);
    if (e != cudaSuccess) return e;
    return launch_pdl(weight_kernel<D>, dim3(2 * D / 8), dim3(kReduceThreads), 0, s,
                      static_cast<const float*>(p.partial), blocks, q_weight ? dq_weight : nullptr,
                      k_weight ? dk_weight : nullptr);
  });
  if (e != cudaSuccess) return cuda_fail(e, "rope gradient launch");
  return ok();
}

}  // extern "C"
