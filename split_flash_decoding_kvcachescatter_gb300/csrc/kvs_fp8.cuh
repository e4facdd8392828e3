// kvs_fp8.cuh -- rows held in 8 bits (e4m3: sign, 4 exponent bits, 3 mantissa
// bits, largest number 448, steps of 2^-9 below 2^-6) with a power of two as the
// scale of each block of 16 positions of a kv head.
//
// Why powers of two: dividing by the scale and growing it later are exact (but
// for what falls under 2^-6 of the stored numbers), so a block's scale and its
// numbers hardly depend on whether its rows came together or one by one, and a
// product with the scale rounds nothing.
#pragma once

#include <cstdint>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

namespace kvs {

constexpr int kScaleBlock = 16;       // positions that share a scale
constexpr int kLeastScaleExp = -60;   // no scale is below 2^-60
constexpr int kMostScaleExp = 100;    // or above 2^100: 448 2^100 leaves room in float32

// The least k with most <= 448 2^k, -60 at least and 100 at most, as 2^k; most >= 0 (a NaN
// counts as 0).
__device__ __forceinline__ float scale_for(float most) {
  const unsigned u = __float_as_uint(most > 0.f ? most : 0.f);
  // most = 1.f 2^e and 448 = 1.75 2^8
  const int k = (int)(u >> 23) - 127 - 8 + ((u & 0x7fffffu) > 0x600000u ? 1 : 0);
  return __uint_as_float((unsigned)(min(max(k, kLeastScaleExp), kMostScaleExp) + 127) << 23);
}

// The larger of most and |x|; an infinity is passed over (0 x is NaN) as NaN is.
__device__ __forceinline__ float finite_max(float most, float x) {
  return fmaxf(most, fmaf(x, 0.f, fabsf(x)));
}

// Two numbers to e4m3 (nearest, ties to even; past 448 they become 448), a in the low byte.
__device__ __forceinline__ unsigned to_e4m3x2(float a, float b) {
  unsigned short r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(b), "f"(a));
  return r;
}
__device__ __forceinline__ unsigned to_e4m3x4(float a, float b, float c, float d) {
  return to_e4m3x2(a, b) | to_e4m3x2(c, d) << 16;
}

// Two e4m3 numbers as float16 (exact), the low byte in the low half.
__device__ __forceinline__ uint32_t from_e4m3x2(uint32_t w) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"((unsigned short)w));
  return r;
}

}  // namespace kvs
