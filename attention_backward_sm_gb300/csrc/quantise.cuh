// Device helpers for rows of bf16 values on their way into a cache: streamed
// loads, and division by a scale with rounding to 8 bits.
#pragma once

#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

namespace fa {

__device__ __forceinline__ float bf_lo(uint32_t u) { return __uint_as_float(u << 16); }
__device__ __forceinline__ float bf_hi(uint32_t u) { return __uint_as_float(u & 0xFFFF0000u); }

// Two values to e4m3 (round to nearest even, saturating to +-448, NaN stays).
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}

__device__ __forceinline__ uint4 ldg_stream(const void* p) {
  uint4 r;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w)
               : "l"(p));
  return r;
}

// A scale and two factors, one below and one above its reciprocal: for any x,
// the fp32 quotient x / s lies between the rounded products x lo and x hi
// (each is off by less than 2^-22 of itself, the factors are 2^-21 apart from
// the reciprocal).  Scales whose reciprocal is out of range get 0 and
// infinity, between which everything lies.  The reciprocal of a power of two
// (of the scale 1 of a cache without scales) is exact and the product with it
// is the quotient, so it is both factors.
struct Scale {
  float s, lo, hi;
  __device__ __forceinline__ explicit Scale(const float* p, int h) : s(p ? *(p + h) : 1.f) {
    const bool plain = s >= 0x1p-100f && s <= 0x1p100f;
    const float inv = 1.f / s, apart = (__float_as_uint(s) & 0x7FFFFFu) == 0 ? 0.f : 0x1p-21f;
    lo = plain ? inv * (1.f - apart) : 0.f;
    hi = plain ? inv * (1.f + apart) : INFINITY;
  }
};

// Eight bf16 values divided by the scale, the quotients rounded to fp32, then
// to e4m3.  Where both products round to the same 8-bit value, so does the
// quotient between them; only where they do not are the divisions carried out
// (5 instructions per value instead of 20).  That is one group of eight in
// 2^13 for a scale with many significant bits, as a largest value over 448
// has.  A scale of few, but no power of two (1.5, 3), puts every 16th value on
// the border of two 8-bit values, and nearly every warp divides: 8191 rows of 16
// heads of 64 10.2 us with 0.0123 or powers of two, 17.6 with 1.5.
__device__ __forceinline__ uint2 quantise8(uint4 x, const Scale& sc) {
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
  uint32_t lo[4], hi[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float a = bf_lo(w[i]), b = bf_hi(w[i]);
    lo[i] = e4m3x2(a * sc.lo, b * sc.lo);
    hi[i] = e4m3x2(a * sc.hi, b * sc.hi);
  }
  uint2 r = make_uint2(lo[0] | lo[1] << 16, lo[2] | lo[3] << 16);
  if (r.x != (hi[0] | hi[1] << 16) || r.y != (hi[2] | hi[3] << 16)) {
#pragma unroll
    for (int i = 0; i < 4; ++i) lo[i] = e4m3x2(__fdiv_rn(bf_lo(w[i]), sc.s), __fdiv_rn(bf_hi(w[i]), sc.s));
    r = make_uint2(lo[0] | lo[1] << 16, lo[2] | lo[3] << 16);
  }
  return r;
}

}  // namespace fa
