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
// a 32-bit product (at position 131072 that would be 0.008 radians).  Of its upper
// 32 bits the first 24 go to sincospif, the rest is a correction of the first order.
//
// All of it is one pass over the rows, bound by HBM: a thread holds 16 values
// of a head (two pieces of 16 bytes that belong together under the rotation),
// d / 16 lanes make a head, and a warp (few tokens: several) goes through the heads
// of a token, whose sines and cosines it works out once and keeps in registers, as
// it does a tensor's weights.  Everything between the loads and the one rounding at
// the end is fp32.
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
constexpr int kMostPairs = 128;
constexpr int kReduceThreads = 256;
constexpr int kMostSms = 152;

__device__ __forceinline__ void load4(const float* from, float2* x) {
  const float4 a = *reinterpret_cast<const float4*>(from);
  x[0] = make_float2(a.x, a.y);
  x[1] = make_float2(a.z, a.w);
}

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
  int rotary;
  int half;              // pairs (i, i + rotary / 2), else (2i, 2i + 1)
  int weight_f32;
  float mscale;
  float sin_scale;       // mscale, or -mscale to turn back
  float eps;
  int num_tokens;
  int split, split_bits; // warps that share a token, and log2 of it
  int heads;
  int heads_kv;
};

// cos and sin of a token, worked out by a warp: c and s of the lane's 8 pairs
// (of the u-th eight).  In shared memory the halves of an eight lie apart, so that
// lanes read them from different banks.
__device__ __forceinline__ void token_turns(const RopeParams& p, const unsigned long long* freqs, int at_position, int u,
                                            float* turns, float2* c, float2* s) {
  const int pairs = p.rotary / 2, lane = threadIdx.x % 32;
  const unsigned long long position = static_cast<unsigned long long>(static_cast<long long>(at_position));
  __syncwarp();   // the token before is done with the place
  for (int i = lane; i < pairs; i += 32) {
    const unsigned long long phase = position * freqs[i];
    // The angle cut off to fp32, and the rest d < 2^-22 radians, with which
    // cos(a + d) = cos a - d sin a.  Of the keys' values in an e4m3 cache 1.8 in 10^6 then
    // fall on the other side of a border than 64-bit arithmetic's (2.9 with the angle
    // rounded to fp32, 1.7 with angles in 64 bits), at the same speed.
    const int half_turns = static_cast<int>(phase >> 32);   // times 2^31
    const float cut = __int2float_rz(half_turns), d = static_cast<float>(half_turns - static_cast<int>(cut)) * (3.14159265f * 0x1p-31f);
    float s0, c0;
    sincospif(cut * 0x1p-31f, &s0, &c0);
    const float sine = fmaf(d, c0, s0), cosine = fmaf(-d, s0, c0);
    const int at = (i >> 2 & 1) * (pairs / 2) + (i >> 3) * 4 + (i & 3);
    turns[at] = cosine * p.mscale;
    turns[kMostPairs + at] = sine * p.sin_scale;
  }
  __syncwarp();
  if (u < pairs / 8) {
    const float* const from = turns + u * 4;
    load4(from, c);
    load4(from + pairs / 2, c + 2);
    load4(from + kMostPairs, s);
    load4(from + kMostPairs + pairs / 2, s + 2);
  }
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

// 8 values, two to a float2.
__device__ __forceinline__ void unpack8(const uint4& v, float2* x) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) x[i] = make_float2(bf_lo(w[i]), bf_hi(w[i]));
}
__device__ __forceinline__ uint4 pack8(const float2* x) {
  return make_uint4(pack_bf16x2(x[0].x, x[0].y), pack_bf16x2(x[1].x, x[1].y), pack_bf16x2(x[2].x, x[2].y),
                    pack_bf16x2(x[3].x, x[3].y));
}
__device__ __forceinline__ uint2 pack8_e4m3(const float2* x) {
  return make_uint2(e4m3x2(x[0].x, x[0].y) | e4m3x2(x[1].x, x[1].y) << 16,
                    e4m3x2(x[2].x, x[2].y) | e4m3x2(x[3].x, x[3].y) << 16);
}
__device__ __forceinline__ float2 both(float x) { return make_float2(x, x); }
// Sum of the products of 16 values with 16 others.
__device__ __forceinline__ float dot16(const float2* x, const float2* y) {
  float2 a = make_float2(0.f, 0.f), b = a;
#pragma unroll
  for (int i = 0; i < 8; i += 2) {
    a = fma2(x[i], y[i], a);
    b = fma2(x[i + 1], y[i + 1], b);
  }
  a = add2(a, b);
  return a.x + a.y;
}
// Positions (and slots) of 32 consecutive tokens, a lane each.
template <bool SLOTS>
struct Tokens {
  int first = 0, position = 0;
  long long slot = 0;
  __device__ __forceinline__ void load(const RopeParams& p, int t) {
    first = t;
    const int at = min(t + static_cast<int>(threadIdx.x % 32), p.num_tokens - 1);
    if (p.rotary > 0) position = p.positions[at];
    if constexpr (SLOTS) slot = p.slots[at];
  }
  __device__ __forceinline__ int lane(const RopeParams& p, int t) {   // t >= first, of the whole warp
    if (t - first >= 32) load(p, t);
    return t - first;
  }
};

// The weights of the lane's 16 values.
__device__ __forceinline__ float weight_at(const void* w, int f32, int i) {
  return f32 ? static_cast<const float*>(w)[i]
             : __uint_as_float(static_cast<uint32_t>(static_cast<const uint16_t*>(w)[i]) << 16);
}
__device__ __forceinline__ void load_weights(const float* weights, const Place& at, float2* x) {
  load4(weights + at.a, x);
  load4(weights + at.a + 4, x + 2);
  load4(weights + at.b, x + 4);
  load4(weights + at.b + 4, x + 6);
}
// What the tokens share, in shared memory: both tensors' weights as fp32 (1 without
// a norm), and the frequencies.
struct Shared {
  unsigned long long freqs[kMostPairs];
  float weights[2 * 256];   // [2][D]
  template <int D>
  __device__ __forceinline__ void stage(const RopeParams& p, bool norm) {   // by the block
    if (norm)
      for (int i = threadIdx.x; i < 2 * D; i += blockDim.x) {
        const void* const w = i < D ? p.q.weight : p.k.weight;
        weights[i] = w ? weight_at(w, p.weight_f32, i % D) : 1.f;
      }
    for (int i = threadIdx.x; i < p.rotary / 2; i += blockDim.x) freqs[i] = p.freqs[i];
  }
};

// x[0..3] is piece a, x[4..7] piece b; c and s of the thread's 8 pairs.
__device__ __forceinline__ void turn16(float2* x, const float2* c, const float2* s, bool half) {
  if (half) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 a = x[i], b = x[4 + i];
      x[i] = fma2(b, make_float2(-s[i].x, -s[i].y), mul2(a, c[i]));
      x[4 + i] = fma2(a, s[i], mul2(b, c[i]));
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float2 a = x[i];
      const float ci = i & 1 ? c[i / 2].y : c[i / 2].x, si = i & 1 ? s[i / 2].y : s[i / 2].x;
      x[i] = make_float2(a.x * ci - a.y * si, a.y * ci + a.x * si);
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
// A pass is 512 / D heads of one tensor of a token: 1 KB, D / 16 lanes a head.  The
// passes of a token are those of its queries, then its keys, then (with a cache) its
// values.

// What a warp keeps of the token and the tensor that it is at.
template <int D, bool NORM, bool CACHE>
struct Forward {
  const RopeParams& p;
  const Place at;
  int t = -1, tensor = -1;
  float2 c[4], s[4], w[NORM ? 8 : 1];
  long long place = -1;   // of the slot in the cache, -1: not in it
  const Shared* shared;   // nullptr: nothing is shared, weights and frequencies come from memory
  Tokens<CACHE> tokens;
  __device__ __forceinline__ Forward(const RopeParams& params, int u, const Shared* sh) : p(params), at(params, u), shared(sh) {}
  __device__ __forceinline__ int heads(int tensor) const { return tensor == 0 ? p.heads : p.heads_kv; }
  __device__ __forceinline__ const uint16_t* row(int tensor, int t) const {
    return tensor == 0 ? p.q.in + t * p.q.in_stride : !CACHE || tensor == 1 ? p.k.in + t * p.k.in_stride : p.v + t * p.v_stride;
  }
  __device__ __forceinline__ void token(int next, int u, float* turns) {
    t = next;
    int position = 0;
    [[maybe_unused]] long long slot = -1;
    if (shared) {
      const int lane = tokens.lane(p, t);
      position = __shfl_sync(0xffffffffu, tokens.position, lane);
      if constexpr (CACHE) slot = __shfl_sync(0xffffffffu, tokens.slot, lane);
    } else {
      if (p.rotary > 0) position = p.positions[t];
      if constexpr (CACHE) slot = p.slots[t];
    }
    token_turns(p, shared ? shared->freqs : p.freqs, position, u, turns, c, s);
    if constexpr (CACHE) {
      const long long num_slots = static_cast<long long>(p.kv.num_pages) * p.kv.page_size;
      place = -1;
      if (slot >= 0 && slot < num_slots) {
        const long long page = slot <= 0x7fffffffll ? p.page_div.quotient(static_cast<int>(slot)) : slot / p.kv.page_size;
        place = page * p.kv.page_stride + (slot - page * p.kv.page_size) * p.kv.slot_stride;
      }
    }
  }
  __device__ __forceinline__ void of(int next) {
    tensor = next;
    if constexpr (NORM) {
      const void* const weight = tensor == 0 ? p.q.weight : p.k.weight;
      if (tensor < 2 && weight) {
        if (shared) {
          load_weights(shared->weights + tensor * D, at, w);
        } else {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            w[i] = make_float2(weight_at(weight, p.weight_f32, at.a + 2 * i), weight_at(weight, p.weight_f32, at.a + 2 * i + 1));
            w[4 + i] = make_float2(weight_at(weight, p.weight_f32, at.b + 2 * i), weight_at(weight, p.weight_f32, at.b + 2 * i + 1));
          }
        }
      }
    }
  }
  // 16 values of head h (there: it exists) to where they belong.
  __device__ __forceinline__ void finish(const uint4& a, const uint4& b, int h, bool there) const {
    if (CACHE && tensor == 2) {
      if (!there || place < 0) return;
      if (p.kv.e4m3) {   // as fa_kv_append stores them
        const Scale sc(p.kv.v_scale, h);
        uint8_t* const to = static_cast<uint8_t*>(p.kv.v) + place + h * p.kv.head_stride;
        *reinterpret_cast<uint2*>(to + at.a) = quantise8(a, sc);
        *reinterpret_cast<uint2*>(to + at.b) = quantise8(b, sc);
      } else {
        uint16_t* const to = static_cast<uint16_t*>(p.kv.v) + place + h * p.kv.head_stride;
        *reinterpret_cast<uint4*>(to + at.a) = a;
        *reinterpret_cast<uint4*>(to + at.b) = b;
      }
      return;
    }
    float2 x[8];
    unpack8(a, x);
    unpack8(b, x + 4);
    if constexpr (NORM) {
      if (tensor == 0 ? p.q.weight != nullptr : p.k.weight != nullptr) {
        const float2 inv = both(rsqrtf(fmaf(head_sum<D>(dot16(x, x)), 1.f / D, p.eps)));
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = mul2(x[i], mul2(inv, w[i]));
      }
    }
    if (at.turned) turn16(x, c, s, p.half);
    if (!there) return;
    if (!CACHE || tensor == 0) {
      uint16_t* const to = (tensor == 0 ? p.q.out + t * p.q.out_stride : p.k.out + t * p.k.out_stride) + h * D;
      *reinterpret_cast<uint4*>(to + at.a) = pack8(x);
      *reinterpret_cast<uint4*>(to + at.b) = pack8(x + 4);
    } else if (place < 0) {
      return;
    } else if (p.kv.e4m3) {
      // Rounded to 8 bits once: the turned values do not pass through bf16.  The product
      // with the rounded reciprocal is off by 2^-23 of the quotient at most, a fraction
      // of the turned values' own fp32 error, so only values that lie that near to the border
      // of two 8-bit ones may take the other (with the rounded quotient the values that
      // differ from 64-bit arithmetic's are as many, and 8191 rows 36.6 -> 37.2 us).
      const Scale sc(p.kv.k_scale, h);
      if (sc.lo > 0.f) {
        const float2 inv = both(__frcp_rn(sc.s));
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = mul2(x[i], inv);
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = make_float2(__fdiv_rn(x[i].x, sc.s), __fdiv_rn(x[i].y, sc.s));
      }
      uint8_t* const to = static_cast<uint8_t*>(p.kv.k) + place + h * p.kv.head_stride;
      *reinterpret_cast<uint2*>(to + at.a) = pack8_e4m3(x);
      *reinterpret_cast<uint2*>(to + at.b) = pack8_e4m3(x + 4);
    } else {
      uint16_t* const to = static_cast<uint16_t*>(p.kv.k) + place + h * p.kv.head_stride;
      *reinterpret_cast<uint4*>(to + at.a) = pack8(x);
      *reinterpret_cast<uint4*>(to + at.b) = pack8(x + 4);
    }
  }
};

// A warp (few tokens: p.split warps) takes the passes of a token, two at a time, the
// first loads before the sines are worked out.  32768 rows of 32 / 8 heads of 128 with
// norms (671 MB): 114 us, 88 % of a copy's rate; 8191 rows of 16 / 4 heads of 64, half
// of each rotated (42 MB): 9.6 us, 65 %; 64 rows of 32 / 8 heads of 128: 3 us, the
// launch and three dependent reads.
template <int D, bool NORM, bool CACHE>
__global__ void __launch_bounds__(kThreads, 3) rope_kernel(const RopeParams p) {
  constexpr int TPH = D / 16, HP = 512 / D;
  __shared__ __align__(16) float turns[kThreads / 32][2 * kMostPairs];
  const int warp = threadIdx.x / 32, u = threadIdx.x % TPH, hl = threadIdx.x % 32 / TPH;
  const long long job = blockIdx.x * static_cast<long long>(kThreads / 32) + warp;
  const long long t_long = job >> p.split_bits;
  const int t = static_cast<int>(t_long), part = static_cast<int>(job) & (p.split - 1);
  pdl_wait();
  if (t_long >= p.num_tokens) return;
  Forward<D, NORM, CACHE> f(p, u, nullptr);
  uint4 a[2], b[2];
  auto load = [&](const uint16_t* row, int heads, int pass) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int h = (pass + i * p.split) * HP + hl;
      a[i] = b[i] = make_uint4(0, 0, 0, 0);
      if (h < heads) {
        a[i] = load16(row + h * D + f.at.a);
        b[i] = load16(row + h * D + f.at.b);
      }
    }
  };
  int before = 0;   // passes of the tensors before, which the warps of a token share in turn
#pragma unroll
  for (int tensor = 0; tensor < (CACHE ? 3 : 2); ++tensor) {
    const int heads = f.heads(tensor), n = (heads + HP - 1) / HP;
    const uint16_t* const row = f.row(tensor, t);
    const int first = (part - before) & (p.split - 1);
    if (first < n) load(row, heads, first);
    if (tensor == 0) f.token(t, u, turns[warp]);
    if (first < n) f.of(tensor);
    for (int pass = first; pass < n; pass += 2 * p.split) {
      if (pass != first) load(row, heads, pass);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        if (pass + i * p.split >= n) break;
        const int h = (pass + i * p.split) * HP + hl;
        f.finish(a[i], b[i], h, h < heads);
      }
    }
    before += n;
  }
}

// Where a warp is in its run of jobs: chunk `chunk` of token t, PASSES passes of one
// tensor each (the last of a tensor may be shorter).
template <int D, int PASSES>
struct Job {
  int t, chunk;
  static constexpr int kHeads = PASSES * (512 / D);
  __device__ __forceinline__ void next(int chunks) {
    if (++chunk == chunks) {
      chunk = 0;
      ++t;
    }
  }
};
__device__ __forceinline__ void bulk_copy(uint32_t dst, const void* src, int bytes, uint32_t bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
               "l"(src), "r"(bytes), "r"(bar)
               : "memory");
}

// Streams: every warp walks through a run of jobs, whose rows come by bulk copies into
// a ring of its own, kRing jobs ahead: what is in flight takes no registers, and 16
// warps keep 192 KB per SM on their way.
constexpr int kRing = 3;
constexpr int kStreamThreads = 512;
constexpr int kStreamWarps = kStreamThreads / 32;
struct Stream {
  static constexpr int kSlot = 4096;   // bytes
  static constexpr int kTurns = kStreamWarps * kRing * kSlot;
  static constexpr int kShared = kTurns + kStreamWarps * 2 * kMostPairs * 4;
  static constexpr int kBars = kShared + sizeof(Shared);
  static constexpr int kMisc = kBars + kStreamWarps * kRing * 8;
  static constexpr int kBytes = kMisc + 16;
};

__device__ int g_rope_status = 0;

// Calls body(job, slot address) for the jobs [first, last) of this warp, once their
// copies, which copy(job, address, barrier) issues, have landed.
template <class J, class Copy, class Body>
__device__ __forceinline__ void stream(uint8_t* smem, J job, long long count, int chunks, Copy copy, Body body) {
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const uint32_t base = smem_u32(smem), slots = base + warp * kRing * Stream::kSlot, bars = base + Stream::kBars + warp * kRing * 8;
  volatile int* const abort = reinterpret_cast<volatile int*>(smem + Stream::kMisc);
  J ahead = job;
  long long asked = 0;
  auto ask = [&](int r) {
    if (asked < count) {
      if (lane == 0) copy(ahead, slots + r * Stream::kSlot, bars + 8 * r);
      ahead.next(chunks);
      ++asked;
    }
  };
  for (int r = 0; r < kRing; ++r) ask(r);
  int r = 0, phase = 0;
  for (long long i = 0; i < count; ++i) {
    const bool ok = mbar_wait(bars + 8 * r, phase, abort, &g_rope_status);
    if (!__all_sync(0xffffffffu, ok)) {
      // what has been asked for lands before the block ends
      volatile int no_abort = 0;
      for (; i < asked; ++i) {
        mbar_wait(bars + 8 * r, phase, &no_abort, &g_rope_status, 100000000ull);
        if (++r == kRing) {
          r = 0;
          phase ^= 1;
        }
      }
      return;
    }
    body(job, slots + r * Stream::kSlot);
    job.next(chunks);
    __syncwarp();   // every lane has read the slot
    ask(r);
    if (++r == kRing) {
      r = 0;
      phase ^= 1;
    }
  }
}

template <int D>
__device__ __forceinline__ void stream_start(const RopeParams& p, uint8_t* smem) {
  if (threadIdx.x == 0) {
    *reinterpret_cast<volatile int*>(smem + Stream::kMisc) = 0;
    for (int i = 0; i < kStreamWarps * kRing; ++i) mbar_init(smem_u32(smem) + Stream::kBars + 8 * i, 1);
    mbar_init_fence();
  }
  pdl_wait();
  reinterpret_cast<Shared*>(smem + Stream::kShared)->stage<D>(p, true);
  __syncthreads();
}
// The run of this warp among so many jobs.
__device__ __forceinline__ void stream_run(long long jobs, long long& first, long long& count) {
  const long long warps = static_cast<long long>(gridDim.x) * kStreamWarps, w = static_cast<long long>(blockIdx.x) * kStreamWarps + threadIdx.x / 32;
  const long long each = jobs / warps, rest = jobs - each * warps;
  first = w * each + min(w, rest);
  count = each + (w < rest ? 1 : 0);
}

__device__ __forceinline__ uint4 lds16(uint32_t at) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(at) : "memory");
  return v;
}

// Many tokens into a cache.  8191 rows of 32 / 8 heads of 128 with norms to e4m3 (185
// MB): 36.6 us, 75 % of a copy's rate (rope_kernel: 43).
template <int D, bool NORM>
__global__ void __launch_bounds__(kStreamThreads, 1) rope_stream_kernel(const RopeParams p) {
  constexpr int TPH = D / 16, HP = 512 / D, PASSES = 4;
  using J = Job<D, PASSES>;
  extern __shared__ __align__(128) uint8_t smem[];
  const int u = threadIdx.x % TPH, hl = threadIdx.x % 32 / TPH;
  float* const turns = reinterpret_cast<float*>(smem + Stream::kTurns) + threadIdx.x / 32 * 2 * kMostPairs;
  stream_start<D>(p, smem);
  Forward<D, NORM, true> f(p, u, reinterpret_cast<const Shared*>(smem + Stream::kShared));
  const int cq = (p.heads + J::kHeads - 1) / J::kHeads, ck = (p.heads_kv + J::kHeads - 1) / J::kHeads;
  const int chunks = cq + 2 * ck;
  long long first, count;
  stream_run(static_cast<long long>(p.num_tokens) * chunks, first, count);
  auto tensor_of = [&](int chunk) { return chunk < cq ? 0 : chunk < cq + ck ? 1 : 2; };
  auto first_head = [&](int chunk, int tensor) { return (chunk - (tensor == 0 ? 0 : tensor == 1 ? cq : cq + ck)) * J::kHeads; };
  J job;
  job.t = static_cast<int>(first / chunks);
  job.chunk = static_cast<int>(first - static_cast<long long>(job.t) * chunks);
  if (count > 0) f.tokens.load(p, job.t);
  stream(smem, job, count, chunks,
         [&](const J& j, uint32_t to, uint32_t bar) {
           const int tensor = tensor_of(j.chunk), h = first_head(j.chunk, tensor), n = min(f.heads(tensor) - h, J::kHeads);
           mbar_arrive_expect_tx(bar, n * D * 2);
           bulk_copy(to, f.row(tensor, j.t) + h * D, n * D * 2, bar);
         },
         [&](const J& j, uint32_t from) {
           if (j.t != f.t) f.token(j.t, u, turns);
           const int tensor = tensor_of(j.chunk), h0 = first_head(j.chunk, tensor), n = min(f.heads(tensor) - h0, J::kHeads);
           if (tensor != f.tensor) f.of(tensor);
#pragma unroll 2
           for (int i = 0; i < n; i += HP) {
             const int h = i + hl;
             const uint32_t row = from + h * D * 2;   // of a head past the last: in the slot, but not used
             const uint4 a = lds16(row + f.at.a * 2), b = lds16(row + f.at.b * 2);
             f.finish(a, b, h0 + h, h < n);
           }
         });
}

// ---------------------------------------------------------------- gradient
// As the stream above, with two rows per job and 16 sums per lane for each weight's
// gradient.  Each block leaves one partial sum per weight; weight_kernel adds them
// in a fixed order.  16384 rows of 16 / 16 heads of 128 (403 MB): 80 us, 75 % of a
// copy's rate; 5001 rows of 8 / 1 heads of 256 (69 MB): 25.9 us, 40 %.  Bound by
// latency: a pass of 1 KB is a chain of 300 instructions (two sums over a head's lanes
// among them), and the 16 warps per SM that the rings and 128 registers leave keep the
// issue slots 44 % busy (38 % at heads of 256).  Without the stores 62 us, without the
// sines 73.
template <int D>
__global__ void __launch_bounds__(kStreamThreads, 1) rope_bwd_kernel(const RopeParams p) {
  constexpr int TPH = D / 16, HP = 512 / D, PASSES = 2;
  using J = Job<D, PASSES>;
  extern __shared__ __align__(128) uint8_t smem[];
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, u = lane % TPH, hl = lane / TPH;
  float* const turns = reinterpret_cast<float*>(smem + Stream::kTurns) + warp * 2 * kMostPairs;
  const Place at(p, u);
  stream_start<D>(p, smem);
  pdl_launch();
  const Shared& shared = *reinterpret_cast<const Shared*>(smem + Stream::kShared);
  float2 acc_q[8], acc_k[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) acc_q[i] = acc_k[i] = make_float2(0.f, 0.f);
  const int cq = (p.heads + J::kHeads - 1) / J::kHeads, chunks = cq + (p.heads_kv + J::kHeads - 1) / J::kHeads;
  long long first, count;
  stream_run(static_cast<long long>(p.num_tokens) * chunks, first, count);
  J job;
  job.t = chunks > 0 ? static_cast<int>(first / chunks) : 0;
  job.chunk = static_cast<int>(first - static_cast<long long>(job.t) * chunks);
  int t = -1, tensor = -1;
  float2 c[4], s[4], w[8];
  const bool q_norm = p.q.weight != nullptr, k_norm = p.k.weight != nullptr;
  bool norm = false;
  uint16_t* to = nullptr;
  Tokens<false> tokens;
  if (count > 0) tokens.load(p, job.t);
  stream(smem, job, count, chunks,
         [&](const J& j, uint32_t to, uint32_t bar) {
           const bool is_q = j.chunk < cq, two = is_q ? q_norm : k_norm;
           const int h = (is_q ? j.chunk : j.chunk - cq) * J::kHeads, n = min((is_q ? p.heads : p.heads_kv) - h, J::kHeads);
           const int bytes = n * D * 2;
           mbar_arrive_expect_tx(bar, two ? 2 * bytes : bytes);
           bulk_copy(to, (is_q ? p.q.in + j.t * p.q.in_stride : p.k.in + j.t * p.k.in_stride) + h * D, bytes, bar);
           if (two)
             bulk_copy(to + Stream::kSlot / 2, (is_q ? p.q.x + j.t * p.q.x_stride : p.k.x + j.t * p.k.x_stride) + h * D, bytes, bar);
         },
         [&](const J& j, uint32_t from) {
           const bool is_q = j.chunk < cq;
           const int h0 = (is_q ? j.chunk : j.chunk - cq) * J::kHeads, n = min((is_q ? p.heads : p.heads_kv) - h0, J::kHeads);
           if (j.t != t) {
             const int at_lane = tokens.lane(p, j.t);
             token_turns(p, shared.freqs, __shfl_sync(0xffffffffu, tokens.position, at_lane), u, turns, c, s);
             tensor = -1;
           }
           t = j.t;
           if (tensor != (is_q ? 0 : 1)) {
             tensor = is_q ? 0 : 1;
             norm = is_q ? q_norm : k_norm;
             to = is_q ? p.q.out + t * p.q.out_stride : p.k.out + t * p.k.out_stride;
             load_weights(shared.weights + (is_q ? 0 : D), at, w);
           }
#pragma unroll
           for (int i = 0; i < PASSES * HP; i += HP) {
             if (i >= n) break;
             const int h = i + hl;
             const uint32_t row = from + h * D * 2;   // of a head past the last: in the slot, but not used
             float2 g[8];
             unpack8(lds16(row + at.a * 2), g);
             unpack8(lds16(row + at.b * 2), g + 4);
             if (at.turned) turn16(g, c, s, p.half);
             if (norm) {
               float2 x[8];
               unpack8(lds16(row + Stream::kSlot / 2 + at.a * 2), x);
               unpack8(lds16(row + Stream::kSlot / 2 + at.b * 2), x + 4);
               const float inv = rsqrtf(fmaf(head_sum<D>(dot16(x, x)), 1.f / D, p.eps));
#pragma unroll
               for (int k = 0; k < 8; ++k) x[k] = mul2(x[k], both(inv));
               if (h < n) {
                 if (is_q) {
#pragma unroll
                   for (int k = 0; k < 8; ++k) acc_q[k] = fma2(g[k], x[k], acc_q[k]);
                 } else {
#pragma unroll
                   for (int k = 0; k < 8; ++k) acc_k[k] = fma2(g[k], x[k], acc_k[k]);
                 }
               }
#pragma unroll
               for (int k = 0; k < 8; ++k) g[k] = mul2(g[k], w[k]);
               const float2 along = both(head_sum<D>(dot16(g, x)) * (-1.f / D));
#pragma unroll
               for (int k = 0; k < 8; ++k) g[k] = mul2(both(inv), fma2(x[k], along, g[k]));
             }
             if (h >= n) continue;
             uint16_t* const row_to = to + (h0 + h) * D;
             *reinterpret_cast<uint4*>(row_to + at.a) = pack8(g);
             *reinterpret_cast<uint4*>(row_to + at.b) = pack8(g + 4);
           }
         });
  // the heads of a warp, then the warps, in order; the rings are free
  float* const sums = reinterpret_cast<float*>(smem);   // [warps][D]
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    float2* const acc = k == 0 ? acc_q : acc_k;
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
      for (int off = TPH; off < 32; off <<= 1) {
        acc[i].x += __shfl_xor_sync(0xffffffffu, acc[i].x, off);
        acc[i].y += __shfl_xor_sync(0xffffffffu, acc[i].y, off);
      }
    __syncthreads();
    if (lane < TPH) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        *reinterpret_cast<float2*>(sums + warp * D + at.a + 2 * i) = acc[i];
        *reinterpret_cast<float2*>(sums + warp * D + at.b + 2 * i) = acc[4 + i];
      }
    }
    __syncthreads();
    for (int i = threadIdx.x; i < D; i += kStreamThreads) {
      float sum = 0.f;
#pragma unroll
      for (int v = 0; v < kStreamWarps; ++v) sum += sums[v * D + i];
      p.partial[(static_cast<long long>(blockIdx.x) * 2 + k) * D + i] = sum;
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
  const int hp = 512 / head_dim, q = (p.heads + hp - 1) / hp, k = (p.heads_kv + hp - 1) / hp;
  const int passes = q + (cache ? 2 : 1) * k, warps = kThreads / 32;
  const bool norm = p.q.weight || p.k.weight;
  // Into a cache, from 8 passes for each of the warps of a stream on, the stream (8191
  // rows of 32 / 8 heads of 128 to e4m3: 36 us, 43 without it; 64 rows: 3.2 us
  // without it, of which its rings would not see a second job).  Rows to rows go
  // without it: 32768 of 32 / 8 heads of 128 with norms 114 us, as a stream 125.
  const bool many = cache && static_cast<long long>(p.num_tokens) * passes >= 8ll * kStreamWarps * dev.sms;
  return with_dim(head_dim, [&](auto d) {
    constexpr int D = decltype(d)::value;
    if (many) {
      static std::atomic<unsigned long long> done[2];
      auto* const kernel = norm ? rope_stream_kernel<D, true> : rope_stream_kernel<D, false>;
      cudaError_t e = prepare_once(reinterpret_cast<const void*>(kernel), Stream::kBytes, dev.id, done[norm]);
      if (e != cudaSuccess) return e;
      return launch_pdl(kernel, dim3(dev.sms), dim3(kStreamThreads), Stream::kBytes, s, p);
    }
    auto* const kernel = cache ? (norm ? rope_kernel<D, true, true> : rope_kernel<D, false, true>)
                               : (norm ? rope_kernel<D, true, false> : rope_kernel<D, false, false>);
    // as many warps per token as have two passes each, up to what runs at once
    const int most = 3 * dev.sms;   // blocks
    p.split = 1;
    p.split_bits = 0;
    while (p.split < warps && 2 * p.split < passes && static_cast<long long>(p.num_tokens) * p.split < most * warps) {
      p.split *= 2;
      ++p.split_bits;
    }
    const long long want = (static_cast<long long>(p.num_tokens) * p.split + warps - 1) / warps;
    return launch_pdl(kernel, dim3(static_cast<unsigned>(want)), dim3(kThreads), 0, s, p);
  });
}

}  // namespace

namespace fa {
cudaError_t rope_status_word(int** word) { return cudaGetSymbolAddress(reinterpret_cast<void**>(word), g_rope_status); }

int rope_read_and_clear_status(cudaStream_t s, int* status) {
  int zero = 0;
  cudaError_t e = cudaMemcpyFromSymbolAsync(status, g_rope_status, sizeof(int), 0, cudaMemcpyDeviceToHost, s);
  if (e == cudaSuccess) e = cudaMemcpyToSymbolAsync(g_rope_status, &zero, sizeof(int), 0, cudaMemcpyHostToDevice, s);
  if (e == cudaSuccess) e = cudaStreamSynchronize(s);
  return static_cast<int>(e);
}
}  // namespace fa

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
  return static_cast<size_t>(kMostSms) * 2 * head_dim * sizeof(float);
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
  // Without tokens only the weights' gradients are written; positions and freqs, which
  // may then be NULL, are not read.
  if (num_tokens == 0) p.rotary = 0;
  p.q.x = q, p.q.x_stride = q_row_stride;
  p.k.x = k, p.k.x_stride = k_row_stride;
  p.partial = static_cast<float*>(workspace);
  const int most = dev.sms < kMostSms ? dev.sms : kMostSms, hp = 512 / head_dim;
  // a job for every warp at least; without tokens the weights' gradients are 0
  const long long jobs = static_cast<long long>(num_tokens) * ((heads + 2 * hp - 1) / (2 * hp) + (heads_kv + 2 * hp - 1) / (2 * hp));
  const long long want = (jobs + kStreamWarps - 1) / kStreamWarps;
  const int blocks = want < 1 ? 1 : want < most ? static_cast<int>(want) : most;
  cudaError_t e = with_dim(head_dim, [&](auto d) {
    constexpr int D = decltype(d)::value;
    static std::atomic<unsigned long long> done{0};
    cudaError_t e = prepare_once(reinterpret_cast<const void*>(rope_bwd_kernel<D>), Stream::kBytes, dev.id, done);
    if (e == cudaSuccess) e = launch_pdl(rope_bwd_kernel<D>, dim3(blocks), dim3(kStreamThreads), Stream::kBytes, s, p);
    if (e != cudaSuccess) return e;
    return launch_pdl(weight_kernel<D>, dim3(2 * D / 8), dim3(kReduceThreads), 0, s,
                      static_cast<const float*>(p.partial), blocks, q_weight ? dq_weight : nullptr,
                      k_weight ? dk_weight : nullptr);
  });
  if (e != cudaSuccess) return cuda_fail(e, "rope gradient launch");
  return ok();
}

}  // extern "C"
