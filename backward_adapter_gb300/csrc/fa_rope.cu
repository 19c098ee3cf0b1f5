// RMS norm of every query and key head with the rotary position in the same pass, and its backward
// (fa_qk_norm_rope, fa_qk_norm_rope_bwd): what turns a projection's output into the q and k of the
// attention entry points, and their gradients back into the projection's.
//
// Work: a row (one head of one token) is read once and written once, bound by HBM. D / 8 lanes hold
// it, each with the two runs of four features that form four rotated pairs, so that a rotation never
// leaves a lane: features 4 l .. and rot / 2 + 4 l .. for pairs (i, i + rot / 2), and 8 l .. 8 l + 7
// for interleaved pairs and for the features that are not rotated. Such a group of lanes stays with
// one token for several heads, which share the token's cosines and sines.
//
// Angles: t = p * f for whole positions p. In turns, f / 2 pi is a fixed-point fraction F of 64 bits
// and p * F modulo 2^64 is the angle modulo a turn, without any rounding that grows with p.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cmath>
#include <type_traits>

#include "fa_check.h"
#include "fa_device.cuh"
#include "tc_ptx.cuh"

namespace fa {
namespace {

struct RopeShape {
  int B, S, Hq, Hkv;
  int half;             // rotated pairs
  int interleaved;
  float eps, factor;
  long long offset, pos_stride_b;
  int chunk;            // heads a group takes
  int q_chunks;         // blockIdx.y below it: queries; above: keys
};

struct RopeArgs {
  RopeShape s;
  RowView x[2];         // q, k
  RowView y[2];         // forward: outputs; backward: gradients of the inputs
  RowView g[2];         // backward: gradients of the outputs
  const void* w[2];
  const float* inv_freq;
  const int64_t* positions;
  float* dw;            // backward: partial weight gradients [2][blocks][D]
};

__device__ __forceinline__ void load4(const float* p, float* x) {
  const float4 a = __ldg(reinterpret_cast<const float4*>(p));
  x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
}
__device__ __forceinline__ void load4(const __nv_bfloat16* p, float* x) {
  const uint2 a = __ldg(reinterpret_cast<const uint2*>(p));
  x[0] = __uint_as_float(a.x << 16);
  x[1] = __uint_as_float(a.x & 0xffff0000u);
  x[2] = __uint_as_float(a.y << 16);
  x[3] = __uint_as_float(a.y & 0xffff0000u);
}
__device__ __forceinline__ void store4(float* p, const float* x) {
  *reinterpret_cast<float4*>(p) = make_float4(x[0], x[1], x[2], x[3]);
}
__device__ __forceinline__ void store4(__nv_bfloat16* p, const float* x) {
  *reinterpret_cast<uint2*>(p) = make_uint2(tc::pack_bf16x2(x[0], x[1]), tc::pack_bf16x2(x[2], x[3]));
}

// f / 2 pi as a 64-bit fraction of a turn (whole turns dropped): f = m 2^e with a 24-bit m, and
// m * floor(2^66 / 2 pi) shifted to the binary point. Off by at most 2^-64 turns.
__device__ __forceinline__ unsigned long long turn_fraction(float f) {
  constexpr unsigned long long k2Pi = 11743562013128004905ull;   // floor(2^66 / (2 pi))
  const uint32_t bits = __float_as_uint(f);
  const int ex = (int)((bits >> 23) & 255u);
  const unsigned long long m = (bits & 0x7fffffu) | (ex != 0 ? 0x800000u : 0u);
  const unsigned long long lo = m * k2Pi, hi = __umul64hi(m, k2Pi);
  const int sh = 152 - (ex != 0 ? ex : 1);                       // e = ex - 150, and the 2 bits of 2^66 / 2^64
  unsigned long long F;
  if (sh <= 0) F = sh > -64 ? lo << -sh : 0;
  else if (sh < 64) F = (lo >> sh) | (hi << (64 - sh));
  else F = sh < 128 ? hi >> (sh - 64) : 0;
  return (bits >> 31) ? 0ull - F : F;
}

template <int N>
__device__ __forceinline__ float group_sum(float x) {
#pragma unroll
  for (int o = N / 2; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}

// What a lane of a token's group needs: where its two runs of features are, and its angles.
template <int D>
struct Lane {
  int c0, c1;
  bool turns;
  float cs[4], sn[4];

  __device__ __forceinline__ Lane(const RopeArgs& a, int l, long long b, int s) {
    const RopeShape& r = a.s;
    turns = 4 * l < r.half;
    c0 = turns && !r.interleaved ? 4 * l : 8 * l;
    c1 = turns && !r.interleaved ? r.half + 4 * l : 8 * l + 4;
#pragma unroll
    for (int j = 0; j < 4; ++j) { cs[j] = 1.f; sn[j] = 0.f; }
    if (!turns) return;
    const long long p = a.positions != nullptr ? __ldg(a.positions + b * r.pos_stride_b + s) : r.offset + s;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const unsigned long long t = (unsigned long long)p * turn_fraction(__ldg(a.inv_freq + 4 * l + j));
      float sine, cosine;   // the top 32 bits, signed: half turns of [-1, 1)
      sincospif((float)(int)(t >> 32) * 4.6566128730773926e-10f, &sine, &cosine);
      cs[j] = cosine * r.factor;
      sn[j] = sine * r.factor;
    }
  }

  // The four pairs are (x[2 j], x[2 j + 1]) when interleaved, (x[j], x[4 + j]) otherwise.
  __device__ __forceinline__ void rotate(float (&x)[8], bool interleaved, float sign) const {
    if (!turns) return;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      float& u = interleaved ? x[2 * j] : x[j];
      float& v = interleaved ? x[2 * j + 1] : x[4 + j];
      const float s = sign * sn[j], p = u, q = v;
      u = p * cs[j] - q * s;
      v = q * cs[j] + p * s;
    }
  }
};

template <typename T, typename W, int D, bool NORM>
__global__ void __launch_bounds__(256) rope_fwd_kernel(RopeArgs a) {
  constexpr int LANES = D / 8, GROUPS = 256 / LANES;
  const int l = threadIdx.x % LANES;
  const long long token = (long long)blockIdx.x * GROUPS + threadIdx.x / LANES;
  const bool on = token < (long long)a.s.B * a.s.S;
  const int s = on ? (int)(token % a.s.S) : 0, b = on ? (int)(token / a.s.S) : 0;
  const int key = (int)blockIdx.y >= a.s.q_chunks;
  const int H = key ? a.s.Hkv : a.s.Hq;
  const int h0 = ((int)blockIdx.y - (key ? a.s.q_chunks : 0)) * a.s.chunk, h1 = min(H, h0 + a.s.chunk);
  const Lane<D> lane(a, l, b, s);
  const bool inter = a.s.interleaved != 0;
  const RowView xv = key ? a.x[1] : a.x[0], yv = key ? a.y[1] : a.y[0];
  const T* x0 = static_cast<const T*>(xv.ptr) + b * xv.sb + s * xv.ss;
  T* y0 = static_cast<T*>(yv.ptr) + b * yv.sb + s * yv.ss;
  float w[8];
  if constexpr (NORM) {
    const W* wp = static_cast<const W*>(key ? a.w[1] : a.w[0]);
    load4(wp + lane.c0, w);
    load4(wp + lane.c1, w + 4);
  }
  for (int h = h0; h < h1; ++h) {
    float x[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    if (on) {
      load4(x0 + h * xv.sh + lane.c0, x);
      load4(x0 + h * xv.sh + lane.c1, x + 4);
    }
    if constexpr (NORM) {
      float sq = 0.f;
#pragma unroll
      for (int j = 0; j < 8; ++j) sq = fmaf(x[j], x[j], sq);
      const float r = rsqrtf(fmaf(group_sum<LANES>(sq), 1.f / D, a.s.eps));
#pragma unroll
      for (int j = 0; j < 8; ++j) x[j] *= r * w[j];
    }
    if (inter) lane.rotate(x, true, 1.f);
    else lane.rotate(x, false, 1.f);
    if (on) {
      store4(y0 + h * yv.sh + lane.c0, x);
      store4(y0 + h * yv.sh + lane.c1, x + 4);
    }
  }
}

// As the forward, with the gradient of the output in and that of the input out. A block adds up its
// rows' weight gradients in registers, then over its groups in shared memory, and writes one row of
// partial sums, which rope_dw_kernel adds in block order.
template <typename T, typename W, int D, bool NORM>
__global__ void __launch_bounds__(256) rope_bwd_kernel(RopeArgs a) {
  constexpr int LANES = D / 8, GROUPS = 256 / LANES;
  const int l = threadIdx.x % LANES, group = threadIdx.x / LANES;
  const int key = (int)blockIdx.y >= a.s.q_chunks;
  const int H = key ? a.s.Hkv : a.s.Hq;
  const int h0 = ((int)blockIdx.y - (key ? a.s.q_chunks : 0)) * a.s.chunk, h1 = min(H, h0 + a.s.chunk);
  const bool inter = a.s.interleaved != 0;
  const RowView xv = key ? a.x[1] : a.x[0], yv = key ? a.y[1] : a.y[0], gv = key ? a.g[1] : a.g[0];
  const long long tokens = (long long)a.s.B * a.s.S;
  float dw[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  int c0 = 0, c1 = 0;
  for (long long t0 = (long long)blockIdx.x * GROUPS; t0 < tokens; t0 += (long long)gridDim.x * GROUPS) {
    const long long token = t0 + group;
    const bool on = token < tokens;
    const int s = on ? (int)(token % a.s.S) : 0, b = on ? (int)(token / a.s.S) : 0;
    const Lane<D> lane(a, l, b, s);
    c0 = lane.c0;
    c1 = lane.c1;
    const T* x0 = static_cast<const T*>(xv.ptr) + b * xv.sb + s * xv.ss;
    const T* g0 = static_cast<const T*>(gv.ptr) + b * gv.sb + s * gv.ss;
    T* y0 = static_cast<T*>(yv.ptr) + b * yv.sb + s * yv.ss;
    float w[8];
    if constexpr (NORM) {
      const W* wp = static_cast<const W*>(key ? a.w[1] : a.w[0]);
      load4(wp + c0, w);
      load4(wp + c1, w + 4);
    }
    for (int h = h0; h < h1; ++h) {
      float g[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f}, x[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
      if (on) {
        load4(g0 + h * gv.sh + c0, g);
        load4(g0 + h * gv.sh + c1, g + 4);
        if constexpr (NORM) {
          load4(x0 + h * xv.sh + c0, x);
          load4(x0 + h * xv.sh + c1, x + 4);
        }
      }
      if (inter) lane.rotate(g, true, -1.f);
      else lane.rotate(g, false, -1.f);
      if constexpr (NORM) {
        float sq = 0.f, tx = 0.f;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          sq = fmaf(x[j], x[j], sq);
          tx = fmaf(g[j] * w[j], x[j], tx);
        }
        sq = group_sum<LANES>(sq);
        tx = group_sum<LANES>(tx);
        const float r = rsqrtf(fmaf(sq, 1.f / D, a.s.eps));
        const float m = tx * (1.f / D) * r * r;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          dw[j] = fmaf(g[j], x[j] * r, dw[j]);
          g[j] = r * fmaf(-x[j], m, g[j] * w[j]);
        }
      }
      if (on) {
        store4(y0 + h * yv.sh + c0, g);
        store4(y0 + h * yv.sh + c1, g + 4);
      }
    }
  }
  if constexpr (NORM) {
    __shared__ float part[GROUPS][D];
    store4(&part[group][c0], dw);
    store4(&part[group][c1], dw + 4);
    __syncthreads();
    for (int d = threadIdx.x; d < D; d += 256) {
      float sum = 0.f;
      for (int i = 0; i < GROUPS; ++i) sum += part[i][d];
      a.dw[((size_t)blockIdx.y * gridDim.x + blockIdx.x) * D + d] = sum;
    }
  }
}

// Adds the blocks' partial weight gradients in order: block 0 the queries' rows, block 1 the keys'.
template <int D>
__global__ void __launch_bounds__(1024) rope_dw_kernel(const float* __restrict__ part, int q_rows, int rows,
                                                       float* __restrict__ dq_w, float* __restrict__ dk_w) {
  constexpr int SLICES = 1024 / D;
  __shared__ float sums[SLICES][D];
  const int first = blockIdx.x ? q_rows : 0, last = blockIdx.x ? rows : q_rows;
  const int d = threadIdx.x % D, slice = threadIdx.x / D;
  float sum = 0.f;
#pragma unroll 8
  for (int i = first + slice; i < last; i += SLICES) sum += part[(size_t)i * D + d];
  sums[slice][d] = sum;
  __syncthreads();
  if (slice != 0) return;
  for (int i = 1; i < SLICES; ++i) sum += sums[i][d];
  float* out = blockIdx.x ? dk_w : dq_w;
  if (out != nullptr) out[d] = sum;
}

// Heads a group of lanes takes, and the grid. More heads share a token's angles; fewer give more
// groups to spread over the SMs.
struct RopeGrid {
  int chunk, q_chunks, k_chunks;
  unsigned x;
};

RopeGrid rope_grid(const RopeShape& s, int D, bool backward) {
  const int groups = 256 / (D / 8);
  const long long blocks = ((long long)s.B * s.S + groups - 1) / groups;
  const long long want = 8LL * sm_count();   // blocks that fill the SMs
  RopeGrid g{16, 0, 0, 0};
  while (g.chunk > 1 && blocks * ((s.Hq + g.chunk - 1) / g.chunk + (s.Hkv + g.chunk - 1) / g.chunk) < want) g.chunk /= 2;
  g.q_chunks = (s.Hq + g.chunk - 1) / g.chunk;
  g.k_chunks = (s.Hkv + g.chunk - 1) / g.chunk;
  long long x = blocks;
  if (backward) {
    const long long most = (want + g.q_chunks + g.k_chunks - 1) / (g.q_chunks + g.k_chunks);
    x = x < most ? x : most;
  }
  g.x = x > 0x7fffffffLL ? 0u : (unsigned)x;
  return g;
}

fa_status check_rope(const fa_rope_params* p, RopeShape& s) {
  clear_error();
  if (p == nullptr) { set_error("params is NULL"); return FA_ERR_INVALID_ARG; }
  if (p->B < 1 || p->B > 65535) { set_error("B=%d outside [1, 65535]", p->B); return FA_ERR_INVALID_ARG; }
  if (p->S < 0 || p->S > kMaxSeq) { set_error("S=%d outside [0, %d]", p->S, kMaxSeq); return FA_ERR_INVALID_ARG; }
  if (p->Hq < 0 || p->Hq > 65535 || p->Hkv < 0 || p->Hkv > 65535 || p->Hq + p->Hkv == 0) {
    set_error("Hq=%d, Hkv=%d: each in [0, 65535], and not both 0", p->Hq, p->Hkv); return FA_ERR_INVALID_ARG;
  }
  if (p->D <= 0) { set_error("D=%d must be positive", p->D); return FA_ERR_INVALID_ARG; }
  if (p->D != 64 && p->D != 128) { set_error("D=%d unsupported (64 or 128)", p->D); return FA_ERR_UNSUPPORTED; }
  if (p->dtype != FA_F32 && p->dtype != FA_BF16) { set_error("dtype=%d invalid", p->dtype); return FA_ERR_INVALID_ARG; }
  if (p->norm != 0 && p->norm != 1) { set_error("norm=%d must be 0 or 1", p->norm); return FA_ERR_INVALID_ARG; }
  if (p->norm && p->w_dtype != FA_F32 && p->w_dtype != p->dtype) {
    set_error("w_dtype=%d: dtype (%d) or FA_F32", p->w_dtype, p->dtype); return FA_ERR_INVALID_ARG;
  }
  if (p->rot < 0 || p->rot > p->D || p->rot % 8 != 0) {
    set_error("rot=%d: a multiple of 8 in [0, %d]", p->rot, p->D); return FA_ERR_INVALID_ARG;
  }
  if (p->interleaved != 0 && p->interleaved != 1) {
    set_error("interleaved=%d must be 0 or 1", p->interleaved); return FA_ERR_INVALID_ARG;
  }
  if (p->norm && !(std::isfinite(p->eps) && p->eps > 0)) { set_error("eps must be finite and above 0"); return FA_ERR_INVALID_ARG; }
  if (!std::isfinite(p->factor)) { set_error("factor is not finite"); return FA_ERR_INVALID_ARG; }
  if (p->pos_stride_b < 0 || p->pos_stride_b > ((int64_t)1 << 40)) {
    set_error("pos_stride_b=%lld outside [0, 2^40]", (long long)p->pos_stride_b); return FA_ERR_INVALID_ARG;
  }
  if (p->offset < -((int64_t)1 << 62) || p->offset > ((int64_t)1 << 62)) {
    set_error("offset=%lld outside [-2^62, 2^62]", (long long)p->offset); return FA_ERR_INVALID_ARG;
  }
  if (p->reserved != 0) { set_error("reserved field must be 0"); return FA_ERR_INVALID_ARG; }
  if (too_large(p->B, p->Hq, p->S, p->D) || too_large(p->B, p->Hkv, p->S, p->D)) {
    set_error("a tensor of these shapes would hold more than 2^40 elements"); return FA_ERR_INVALID_ARG;
  }
  s = RopeShape{p->B, p->S, p->Hq, p->Hkv, p->rot / 2, p->interleaved, p->eps, p->factor,
                (long long)p->offset, (long long)p->pos_stride_b, 0, 0};
  return FA_OK;
}

// The small inputs: weights, frequencies and positions; appends their spans.
fa_status check_small(const fa_rope_params* p, const void* q_weight, const void* k_weight, const float* inv_freq,
                      const int64_t* positions, Span* in, int& n) {
  const size_t wb = p->norm ? (size_t)p->D * (p->w_dtype == FA_BF16 ? 2 : 4) : 0;
  in[n++] = {q_weight, p->Hq ? wb : 0, "q_weight"};
  in[n++] = {k_weight, p->Hkv ? wb : 0, "k_weight"};
  if (p->rot > 0 && inv_freq == nullptr) { set_error("inv_freq is NULL"); return FA_ERR_INVALID_ARG; }
  if ((uintptr_t)inv_freq % 4 != 0 || (uintptr_t)positions % 8 != 0) {
    set_error("inv_freq must be 4-byte and positions 8-byte aligned"); return FA_ERR_INVALID_ARG;
  }
  return FA_OK;
}

fa_status check_apart(const Span* out, int n_out, const fa_rope_params* p, const float* inv_freq, const int64_t* positions) {
  const Span in[2] = {{inv_freq, (size_t)p->rot / 2 * 4, "inv_freq"},
                      {positions, ((size_t)(p->B - 1) * p->pos_stride_b + p->S) * 8, "positions"}};
  for (int o = 0; o < n_out; ++o)
    for (const Span& x : in)
      if (overlaps(out[o], x)) { set_error("output %s overlaps input %s", out[o].name, x.name); return FA_ERR_INVALID_ARG; }
  return FA_OK;
}

template <typename F>
void by_type(const fa_rope_params* p, F f) {
  using D64 = std::integral_constant<int, 64>;
  using D128 = std::integral_constant<int, 128>;
  auto by_dim = [&](auto t, auto w) {
    if (p->D == 64) f(t, w, D64{});
    else f(t, w, D128{});
  };
  if (p->dtype == FA_F32) by_dim(float{}, float{});
  else if (p->norm && p->w_dtype == FA_F32) by_dim(__nv_bfloat16{}, float{});
  else by_dim(__nv_bfloat16{}, __nv_bfloat16{});
}

}  // namespace
}  // namespace fa

using namespace fa;

extern "C" {

fa_status fa_qk_norm_rope(const fa_rope_params* p, const fa_view* q, const fa_view* k, const void* q_weight,
                          const void* k_weight, const float* inv_freq, const int64_t* positions, const fa_view* q_out,
                          const fa_view* k_out, void* stream) {
  RopeArgs a{};
  fa_status st = check_rope(p, a.s);
  if (st != FA_OK) return st;
  const size_t es = p->dtype == FA_BF16 ? 2 : 4;
  Span in[4], out[2];
  if ((st = check_view(q, p->B, p->S, p->Hq, p->D, es, false, "q", in[0])) != FA_OK) return st;
  if ((st = check_view(k, p->B, p->S, p->Hkv, p->D, es, false, "k", in[1])) != FA_OK) return st;
  if ((st = check_view(q_out, p->B, p->S, p->Hq, p->D, es, true, "q_out", out[0])) != FA_OK) return st;
  if ((st = check_view(k_out, p->B, p->S, p->Hkv, p->D, es, true, "k_out", out[1])) != FA_OK) return st;
  int n = 2;
  if ((st = check_small(p, q_weight, k_weight, inv_freq, positions, in, n)) != FA_OK) return st;
  if ((st = check_buffers(in, n, out, 2)) != FA_OK) return st;
  if ((st = check_apart(out, 2, p, inv_freq, positions)) != FA_OK) return st;
  if (p->S == 0) return FA_OK;
  const RopeGrid g = rope_grid(a.s, p->D, false);
  if (g.x == 0 || g.q_chunks + g.k_chunks > 65535) { set_error("too many rows for one launch"); return FA_ERR_UNSUPPORTED; }
  a.s.chunk = g.chunk;
  a.s.q_chunks = g.q_chunks;
  a.x[0] = row_view(q); a.x[1] = row_view(k);
  a.y[0] = row_view(q_out); a.y[1] = row_view(k_out);
  a.w[0] = q_weight; a.w[1] = k_weight;
  a.inv_freq = inv_freq;
  a.positions = positions;
  const dim3 grid(g.x, (unsigned)(g.q_chunks + g.k_chunks));
  cudaStream_t cs = (cudaStream_t)stream;
  by_type(p, [&](auto t, auto w, auto dim) {
    using T = decltype(t);
    using W = decltype(w);
    constexpr int D = decltype(dim)::value;
    if (p->norm) rope_fwd_kernel<T, W, D, true><<<grid, 256, 0, cs>>>(a);
    else if constexpr (std::is_same_v<T, W>) rope_fwd_kernel<T, T, D, false><<<grid, 256, 0, cs>>>(a);
  });
  count_launches(1);
  return cuda_status(cudaGetLastError(), "norm and rotation launch");
}

size_t fa_qk_norm_rope_bwd_workspace_size(const fa_rope_params* p) {
  RopeShape s;
  if (check_rope(p, s) != FA_OK || !p->norm || p->S == 0) return 0;
  const RopeGrid g = rope_grid(s, p->D, true);
  return align_up((size_t)g.x * (g.q_chunks + g.k_chunks) * p->D * 4);
}

fa_status fa_qk_norm_rope_bwd(const fa_rope_params* p, const fa_view* dq_out, const fa_view* dk_out, const fa_view* q,
                              const fa_view* k, const void* q_weight, const void* k_weight, const float* inv_freq,
                              const int64_t* positions, const fa_view* dq, const fa_view* dk, float* dq_weight,
                              float* dk_weight, void* ws, size_t ws_bytes, void* stream) {
  RopeArgs a{};
  fa_status st = check_rope(p, a.s);
  if (st != FA_OK) return st;
  const size_t es = p->dtype == FA_BF16 ? 2 : 4;
  Span in[6], out[4];
  if ((st = check_view(dq_out, p->B, p->S, p->Hq, p->D, es, false, "dq_out", in[0])) != FA_OK) return st;
  if ((st = check_view(dk_out, p->B, p->S, p->Hkv, p->D, es, false, "dk_out", in[1])) != FA_OK) return st;
  in[2] = {nullptr, 0, "q"};
  in[3] = {nullptr, 0, "k"};
  if (p->norm) {
    if ((st = check_view(q, p->B, p->S, p->Hq, p->D, es, false, "q", in[2])) != FA_OK) return st;
    if ((st = check_view(k, p->B, p->S, p->Hkv, p->D, es, false, "k", in[3])) != FA_OK) return st;
  }
  if ((st = check_view(dq, p->B, p->S, p->Hq, p->D, es, true, "dq", out[0])) != FA_OK) return st;
  if ((st = check_view(dk, p->B, p->S, p->Hkv, p->D, es, true, "dk", out[1])) != FA_OK) return st;
  out[2] = {dq_weight, p->norm && p->Hq ? (size_t)p->D * 4 : 0, "dq_weight"};
  out[3] = {dk_weight, p->norm && p->Hkv ? (size_t)p->D * 4 : 0, "dk_weight"};
  int n = 4;
  if ((st = check_small(p, q_weight, k_weight, inv_freq, positions, in, n)) != FA_OK) return st;
  if ((st = check_buffers(in, n, out, 4)) != FA_OK) return st;
  if ((st = check_apart(out, 4, p, inv_freq, positions)) != FA_OK) return st;
  cudaStream_t cs = (cudaStream_t)stream;
  const size_t need = fa_qk_norm_rope_bwd_workspace_size(p);
  Span all[10];
  for (int i = 0; i < n; ++i) all[i] = in[i];
  for (int i = 0; i < 4; ++i) all[n + i] = out[i];
  if ((st = check_ws(ws, ws_bytes, need, all, n + 4)) != FA_OK) return st;
  if (p->S == 0) {   // no rows: the weights' gradient is zero
    cudaError_t e = out[2].n ? cudaMemsetAsync(dq_weight, 0, out[2].n, cs) : cudaSuccess;
    if (e == cudaSuccess && out[3].n) e = cudaMemsetAsync(dk_weight, 0, out[3].n, cs);
    return cuda_status(e, "zero weight gradients");
  }
  const RopeGrid g = rope_grid(a.s, p->D, true);
  if (g.x == 0 || g.q_chunks + g.k_chunks > 65535) { set_error("too many rows for one launch"); return FA_ERR_UNSUPPORTED; }
  a.s.chunk = g.chunk;
  a.s.q_chunks = g.q_chunks;
  a.x[0] = row_view(q); a.x[1] = row_view(k);
  a.y[0] = row_view(dq); a.y[1] = row_view(dk);
  a.g[0] = row_view(dq_out); a.g[1] = row_view(dk_out);
  a.w[0] = q_weight; a.w[1] = k_weight;
  a.inv_freq = inv_freq;
  a.positions = positions;
  a.dw = static_cast<float*>(ws);
  const dim3 grid(g.x, (unsigned)(g.q_chunks + g.k_chunks));
  by_type(p, [&](auto t, auto w, auto dim) {
    using T = decltype(t);
    using W = decltype(w);
    constexpr int D = decltype(dim)::value;
    if (p->norm) rope_bwd_kernel<T, W, D, true><<<grid, 256, 0, cs>>>(a);
    else if constexpr (std::is_same_v<T, W>) rope_bwd_kernel<T, T, D, false><<<grid, 256, 0, cs>>>(a);
  });
  count_launches(1);
  cudaError_t e = cudaGetLastError();
  if (e == cudaSuccess && p->norm) {
    const int q_rows = (int)g.x * g.q_chunks, rows = q_rows + (int)g.x * g.k_chunks;
    if (p->D == 64) rope_dw_kernel<64><<<2, 1024, 0, cs>>>(a.dw, q_rows, rows, p->Hq ? dq_weight : nullptr, p->Hkv ? dk_weight : nullptr);
    else rope_dw_kernel<128><<<2, 1024, 0, cs>>>(a.dw, q_rows, rows, p->Hq ? dq_weight : nullptr, p->Hkv ? dk_weight : nullptr);
    count_launches(1);
    e = cudaGetLastError();
  }
  return cuda_status(e, "norm and rotation backward launch");
}

}  // extern "C"
