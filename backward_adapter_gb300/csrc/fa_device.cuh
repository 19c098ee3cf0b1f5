// Small device helpers shared by the kernels: element loads/stores and the
// per-pair visibility rule of the op.
#pragma once

#include <cuda_bf16.h>
#include <math_constants.h>
#include <stdint.h>

#include "fa_internal.h"

namespace fa {

__device__ __forceinline__ float to_f(float x) { return x; }
__device__ __forceinline__ float to_f(__nv_bfloat16 x) { return __bfloat162float(x); }

__device__ __forceinline__ void from_f(float* p, float x) { *p = x; }
__device__ __forceinline__ void from_f(__nv_bfloat16* p, float x) { *p = __float2bfloat16_rn(x); }

__device__ __forceinline__ float warp_sum(float x) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}

__device__ __forceinline__ float warp_max(float x) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, o));
  return x;
}

// Programmatic dependent launch: a kernel launched by launch_after may start while the one before it in
// the stream still runs, once every block of that one has called let_next_kernel_start (or ended); what
// it does before wait_for_kernel_before must not touch what the other writes. The wait ends when the
// kernel before has finished and its writes are visible.
__device__ __forceinline__ void let_next_kernel_start() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void wait_for_kernel_before() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

template <typename... P, typename... A>
cudaError_t launch_after(void (*kernel)(P...), dim3 grid, int threads, cudaStream_t st, A... args) {
  cudaLaunchAttribute at{};
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t c{};
  c.gridDim = grid;
  c.blockDim = dim3(threads);
  c.stream = st;
  c.attrs = &at;
  c.numAttrs = 1;
  return cudaLaunchKernelEx(&c, kernel, P(args)...);
}

// Threshold at and below which an additive mask value hides a pair (the
// "mask floor" of the tiled backward in llama.cpp PR #57, commit 86c140d).
constexpr float kMaskFloor = -1e9f;

// Whether query row i may attend to key j, and the additive bias of the pair.
// Rows/keys outside [0, Sq) x [0, Sk) are invisible.
__device__ __forceinline__ bool pair_visible(const Shape& s, const void* mask, int b, int i, int j,
                                             float& bias) {
  bias = 0.f;
  if (i >= s.Sq || j >= s.Sk) return false;
  if (s.causal && (long long)j > s.q_offset + i) return false;
  if (s.window > 0 && llabs(s.q_offset + i - (long long)j) > s.window) return false;
  if (s.mask_kind != MK_NONE) {
    const size_t mb = (s.mask_batch > 1) ? (size_t)b : 0;
    const size_t idx = (mb * (size_t)s.Sq + (size_t)i) * (size_t)s.Sk + (size_t)j;
    if (s.mask_kind == MK_ADD) {
      const float m = static_cast<const float*>(mask)[idx];
      if (!(m > kMaskFloor)) return false;
      bias = m;
    } else {
      if (static_cast<const uint8_t*>(mask)[idx] == 0) return false;
    }
  }
  return true;
}

}  // namespace fa
