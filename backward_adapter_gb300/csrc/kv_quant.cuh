// The blocks of a quantized K/V cache (q8_0, q4_0): storing 32 features as an fp16 scale and 8- or
// 4-bit numbers, and their values. Four consecutive lanes hold a block when it is written, 8
// features each.
#pragma once

#include <cuda_fp16.h>
#include <math_constants.h>
#include <stdint.h>

#include "kv_q8.cuh"

namespace fa {

constexpr float kFp16Max = 65504.0f;

// What a block stores of x: not-a-number as 0, infinities as the largest finite number.
__device__ __forceinline__ float storable(float x) {
  return x == x ? fminf(fmaxf(x, -CUDART_MAX_NORMAL_F), CUDART_MAX_NORMAL_F) : 0.f;
}

// Quantizes the block that this lane and the three others of its aligned group of four hold (all 32
// lanes of the warp call it). Returns the block's scale (the same in the four lanes) and this
// lane's 8 numbers, one per byte: q (q8_0) or q + 8 (q4_0). The scale is rounded to fp16 before
// the division, so that a value is off by at most half of the step that is stored; the division
// and the rounding are exact in fp32, which makes the numbers those of the definition.
template <bool Q4>
__device__ __forceinline__ __half quantize_block(float (&x)[8], uint32_t& lo, uint32_t& hi) {
  float top = 0.f;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    x[j] = storable(x[j]);
    top = fmaxf(top, fabsf(x[j]));
  }
  const float own = top;
  top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
  top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
  __half d;
  if constexpr (Q4) {
    // the signed value of largest magnitude; of equal ones the lowest index: the lowest lane that
    // holds one, and its first
    float m = 0.f;
#pragma unroll
    for (int j = 7; j >= 0; --j)
      if (fabsf(x[j]) == top) m = x[j];
    const unsigned first = (threadIdx.x & 31u) & ~3u;
    const unsigned has = (__ballot_sync(0xffffffffu, own == top) >> first) & 15u;
    m = __shfl_sync(0xffffffffu, m, (int)first + __ffs(has) - 1);
    d = __float2half_rn(fminf(fmaxf(m * -0.125f, -kFp16Max), kFp16Max));
  } else {
    d = __float2half_rn(fminf(__fdiv_rn(top, 127.0f), kFp16Max));
  }
  const float df = __half2float(d);
  const float low = Q4 ? -8.f : -127.f, high = Q4 ? 7.f : 127.f;
  lo = hi = 0;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const float r = df != 0.f ? fminf(fmaxf(rintf(__fdiv_rn(x[j], df)), low), high) : 0.f;
    const uint32_t n = (uint32_t)((int)r + (Q4 ? 8 : 0)) & 0xffu;
    if (j < 4) lo |= n << (8 * j);
    else hi |= n << (8 * (j - 4));
  }
  return d;
}

}  // namespace fa
