// The blocks of a quantized K/V cache (q8_0, q4_0): storing 32 features as an fp16 scale and 8- or
// 4-bit numbers. Two neighbouring lanes hold a block when it is written, 16 features each.
#pragma once

#include <cuda_fp16.h>
#include <math_constants.h>
#include <stdint.h>

#include "kv_q8.cuh"
#include "tc_ptx.cuh"

namespace fa {

constexpr float kFp16Max = 65504.0f;

// What a block stores of x: not-a-number as 0, infinities as the largest finite number.
__device__ __forceinline__ float storable(float x) {
  return x == x ? fminf(fmaxf(x, -CUDART_MAX_NORMAL_F), CUDART_MAX_NORMAL_F) : 0.f;
}

// Quantizes half a block, 16 features: this lane's, an even one's the first (all 32 lanes of the warp call it). Returns the
// block's scale (the same in both lanes) and this lane's 16 numbers, one per byte: q (q8_0) or q + 8 (q4_0). The scale is
// rounded to fp16 before the division, so that a value is off by at most half of the step that is stored; the division
// and the rounding are exact in fp32, which makes the numbers those of the definition.
//
// One reciprocal serves a block: with r = 1 / d correctly rounded and y = x r, y + (x - y d) r in fused operations is x / d
// correctly rounded (Markstein, Computation of elementary functions on the IBM RISC System/6000, 1990; d has 11 bits, so it is
// not the exception, a significand of ones). Scales below 2^-14, which have fewer bits, and those held to the largest fp16 are
// divided by: elsewhere no quotient is beyond 127 (8 in 4 bits) once rounded.
template <bool Q4>
__device__ __forceinline__ __half quantize_half_block(float (&x)[16], uint32_t (&w)[4]) {
  uint64_t odd = 0;   // not-a-numbers and infinities times 0
#pragma unroll
  for (int j = 0; j < 16; j += 2) odd = tc::fma_f32x2(tc::f32x2(x[j], x[j + 1]), 0, odd);
  float odd_lo, odd_hi;
  tc::f32x2_split(odd, odd_lo, odd_hi);
  if (!(odd_lo + odd_hi == 0.f)) {
#pragma unroll
    for (int j = 0; j < 16; ++j) x[j] = storable(x[j]);
  }
  float most = x[0], least = x[0];
#pragma unroll
  for (int j = 1; j < 16; ++j) {
    most = fmaxf(most, x[j]);
    least = fminf(least, x[j]);
  }
  most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, 1));
  least = fminf(least, __shfl_xor_sync(0xffffffffu, least, 1));
  __half d;
  if constexpr (Q4) {
    // the signed value of largest magnitude; of equal ones the lowest index
    float m = most > -least ? most : least;
    const bool equal = most == -least;
    if (__any_sync(0xffffffffu, equal)) {
      float own = 0.f;
      bool has = false;
#pragma unroll
      for (int j = 15; j >= 0; --j)
        if (fabsf(x[j]) == most) {
          own = x[j];
          has = true;
        }
      const float other = __shfl_xor_sync(0xffffffffu, own, 1);
      const bool others = __shfl_xor_sync(0xffffffffu, (int)has, 1) != 0;
      if (equal) m = (threadIdx.x & 1) == 0 ? (has ? own : other) : (others ? other : own);
    }
    d = __float2half_rn(fminf(fmaxf(m * -0.125f, -kFp16Max), kFp16Max));
  } else {
    d = __float2half_rn(fminf(__fdiv_rn(fmaxf(most, -least), 127.0f), kFp16Max));
  }
  const float df = __half2float(d);
  const float inv = __frcp_rn(df);
  // 1.5 * 2^23: a sum with it has the nearest whole number in its low bits; 4 bits' numbers are 8 more
  constexpr float kRound = Q4 ? 12582920.f : 12582912.f;
  const uint64_t r = tc::f32x2(inv, inv), less_d = tc::f32x2(-df, -df), up = tc::f32x2(kRound, kRound);
  float n[16];
#pragma unroll
  for (int j = 0; j < 16; j += 2) {
    const uint64_t xx = tc::f32x2(x[j], x[j + 1]);
    uint64_t y = tc::mul_f32x2(xx, r);
    y = tc::fma_f32x2(tc::fma_f32x2(y, less_d, xx), r, y);
    tc::f32x2_split(tc::add_f32x2(y, up), n[j], n[j + 1]);
  }
  const float size = fabsf(df);
  if (size < 6.103515625e-5f || size >= kFp16Max) {
    const float low = Q4 ? -8.f : -127.f, high = Q4 ? 7.f : 127.f;
#pragma unroll
    for (int j = 0; j < 16; ++j)
      n[j] = kRound + (df != 0.f ? fminf(fmaxf(rintf(__fdiv_rn(x[j], df)), low), high) : 0.f);
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {   // the low bytes
    const float* v = n + 4 * i;
    w[i] = __byte_perm(__byte_perm(__float_as_uint(v[0]), __float_as_uint(v[1]), 0x0040),
                       __byte_perm(__float_as_uint(v[2]), __float_as_uint(v[3]), 0x0040), 0x5410);
    if constexpr (Q4) w[i] -= (w[i] >> 4) & 0x01010101u;   // 16 is held to 15
  }
  return d;
}

}  // namespace fa
