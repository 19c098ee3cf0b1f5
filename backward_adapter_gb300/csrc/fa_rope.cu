// RMS norm of every query and key head with the rotary position in the same pass, and its backward
// (fa_qk_norm_rope, fa_qk_norm_rope_bwd): what turns a projection's output into the q and k of the
// attention entry points, and their gradients back into the projection's.
//
// Work: a row (one head of one token) is read once and written once, bound by HBM. D / (2 E) lanes hold
// it, each with the two runs of E features that form E rotated pairs, so that a rotation never leaves a
// lane: features E l .. and rot / 2 + E l .. for pairs (i, i + rot / 2), and 2 E l .. for interleaved
// pairs and for the features that are not rotated. E is 8 for many rows of bf16 (see run_of), else 4.
// Such a group of lanes stays with one token for several heads, which share the token's cosines and
// sines. The next heads' rows are on their way to a ring in shared memory meanwhile, each lane's bytes in
// slots of its own (cp.async; nothing to wait for but one's own copies): held in registers they would
// cost the occupancy that hides their latency. Next to HBM instructions are the bound, so products and sums run on packed
// pairs of fp32.
//
// Measured (device time, captured calls over changing inputs), bf16, D = 128, 32 + 8 heads: 4 x 4096 tokens forward 54.0 us,
// 6.2 TB/s, 92% of the measured copy rate; 2 x 4096 tokens backward 45.3 us with the weights' sums, 82% (at 4 x 4096
// 94%: the sums' kernel and the ramps are a fixed 6 us); one token of 8 sequences 2.5 us, a launch. fp32, 4 x 4096 tokens:
// forward 98.8 us and backward 147.7, the copy rate.
//
// Angles: t = p * f for whole positions p. In turns, f / 2 pi is a fixed-point fraction F of 64 bits, off by at most
// (1 + |f| / 4) 2^-64, and p * F modulo 2^64 is the angle modulo a turn: off by |p| times that, and by 2^-32 turns where it is cut to
// 32 bits for sine and cosine. For |p| below 2^31 and frequencies up to 1 both together are below 2^-31 turns.
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

// E consecutive features as they are in memory, their values, and back.
template <typename T, int E>
struct Run {
  static constexpr int BYTES = E * sizeof(T), UNIT = BYTES < 16 ? BYTES : 16, UNITS = BYTES / UNIT;
  uint32_t u[BYTES / 4];
  __device__ __forceinline__ void load(const T* p) {
#pragma unroll
    for (int i = 0; i < BYTES / 8; ++i) {
      const uint2 a = __ldg(reinterpret_cast<const uint2*>(p) + i);
      u[2 * i] = a.x; u[2 * i + 1] = a.y;
    }
  }
  // The run's units are 256 * UNIT bytes apart in shared memory, the threads' side by side.
  __device__ __forceinline__ static void copy(uint32_t slot, const T* p) {
#pragma unroll
    for (int i = 0; i < UNITS; ++i) {
      const char* src = reinterpret_cast<const char*>(p) + i * UNIT;
      if constexpr (UNIT == 16)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(slot + i * 256 * UNIT), "l"(src) : "memory");
      else
        asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(slot + i * 256 * UNIT), "l"(src) : "memory");
    }
  }
  __device__ __forceinline__ void fetch(uint32_t slot) {
#pragma unroll
    for (int i = 0; i < UNITS; ++i) {
      uint32_t* v = u + i * UNIT / 4;
      if constexpr (UNIT == 16)
        asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]) : "r"(slot + i * 256 * UNIT) : "memory");
      else
        asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(v[0]), "=r"(v[1]) : "r"(slot + i * 256 * UNIT) : "memory");
    }
  }
  // As pairs of consecutive features.
  __device__ __forceinline__ void values(uint64_t* x) const {
#pragma unroll
    for (int i = 0; i < E / 2; ++i) {
      if constexpr (sizeof(T) == 4) x[i] = tc::f32x2(__uint_as_float(u[2 * i]), __uint_as_float(u[2 * i + 1]));
      else x[i] = tc::f32x2(__uint_as_float(u[i] << 16), __uint_as_float(u[i] & 0xffff0000u));
    }
  }
  __device__ __forceinline__ void store(T* p, const uint64_t* x) {
#pragma unroll
    for (int i = 0; i < E / 2; ++i) {
      float lo, hi;
      tc::f32x2_split(x[i], lo, hi);
      if constexpr (sizeof(T) == 4) {
        u[2 * i] = __float_as_uint(lo);
        u[2 * i + 1] = __float_as_uint(hi);
      } else {
        u[i] = tc::pack_bf16x2(lo, hi);
      }
    }
    if constexpr (UNIT == 16) {
#pragma unroll
      for (int i = 0; i < UNITS; ++i)
        reinterpret_cast<uint4*>(p)[i] = make_uint4(u[4 * i], u[4 * i + 1], u[4 * i + 2], u[4 * i + 3]);
    } else {
      *reinterpret_cast<uint2*>(p) = make_uint2(u[0], u[1]);
    }
  }
};

// f / 2 pi as a 64-bit fraction of a turn (whole turns dropped): f = m 2^e with a 24-bit m, and
// m * floor(2^66 / 2 pi) shifted to the binary point. Off by less than a step, 2^-64 turns, for what the shift drops, and by
// f / 4 steps for what the constant lacks (less than one in its last place, times m).
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
template <int E, bool INTER>
struct Lane {
  int c0, c1;
  bool turns;
  float cs[E], sn[E];

  __device__ __forceinline__ Lane(const RopeArgs& a, int l) {
    turns = E * l < a.s.half;
    c0 = turns && !INTER ? E * l : 2 * E * l;
    c1 = turns && !INTER ? a.s.half + E * l : 2 * E * l + E;
  }
  __device__ __forceinline__ void angles(const RopeArgs& a, int l, long long b, int s) {
    if (!turns) return;
    const RopeShape& r = a.s;
    const long long p = a.positions != nullptr ? __ldg(a.positions + b * r.pos_stride_b + s) : r.offset + s;
#pragma unroll
    for (int j = 0; j < E; ++j) {
      const float f = __ldg(a.inv_freq + E * l + j);
      const unsigned long long t = (unsigned long long)p * turn_fraction(f);
      // the top 32 bits, signed: half turns of [-1, 1)
      sincospif((float)(int)(t >> 32) * 4.6566128730773926e-10f, &sn[j], &cs[j]);
      const float by = r.factor + (f - f);   // not a number where f is infinite or none
      cs[j] *= by;
      sn[j] *= by;
    }
  }

};

__device__ __forceinline__ uint64_t twice(float x) { return tc::f32x2(x, x); }
__device__ __forceinline__ uint64_t swapped(uint64_t x) {
  float lo, hi;
  tc::f32x2_split(x, lo, hi);
  return tc::f32x2(hi, lo);
}
__device__ __forceinline__ float both(uint64_t x) {
  float lo, hi;
  tc::f32x2_split(x, lo, hi);
  return lo + hi;
}

// The rotation of a lane's 2 E features, held as E pairs of neighbours x: the rotated pairs (p, q) are the neighbours
// themselves when interleaved, else neighbours of x[i] with those of x[E / 2 + i]. In both cases
// x'[i] = x[i] * a[i] + (what x[i] turns with) * b[i], packed.
template <int E, bool INTER>
struct Turn {
  uint64_t a[E], b[E];

  // By the lane's angles, or back; each feature times its weight first (w: as x).
  template <bool BACK>
  __device__ __forceinline__ Turn(const Lane<E, INTER>& l, const uint64_t (&w)[E], std::bool_constant<BACK>) {
#pragma unroll
    for (int i = 0; i < E; ++i) {
      a[i] = w[i];   // all there is to a lane that does not turn
      b[i] = 0;
      if (!l.turns) continue;
      if constexpr (INTER) {
        const float s = BACK ? -l.sn[i] : l.sn[i];
        a[i] = tc::mul_f32x2(w[i], twice(l.cs[i]));
        b[i] = tc::mul_f32x2(swapped(w[i]), tc::f32x2(-s, s));
      } else {
        const int j = i % (E / 2), other = i < E / 2 ? E / 2 + j : j;
        const float s0 = (i < E / 2) != BACK ? -l.sn[2 * j] : l.sn[2 * j];
        const float s1 = (i < E / 2) != BACK ? -l.sn[2 * j + 1] : l.sn[2 * j + 1];
        a[i] = tc::mul_f32x2(w[i], tc::f32x2(l.cs[2 * j], l.cs[2 * j + 1]));
        b[i] = tc::mul_f32x2(w[other], tc::f32x2(s0, s1));
      }
    }
  }
  __device__ __forceinline__ void operator()(uint64_t (&x)[E]) const {
    uint64_t y[E];
#pragma unroll
    for (int i = 0; i < E; ++i) {
      const uint64_t with = INTER ? swapped(x[i]) : x[i < E / 2 ? E / 2 + i : i - E / 2];
      y[i] = tc::fma_f32x2(with, b[i], tc::mul_f32x2(x[i], a[i]));
    }
#pragma unroll
    for (int i = 0; i < E; ++i) x[i] = y[i];
  }
};

// Heads on their way for each lane, and the ring that holds them (n tensors).
constexpr int kAhead = 4;
template <typename T, int E>
constexpr int ring_bytes(int n) { return kAhead * n * 2 * Run<T, E>::BYTES * 256; }

template <typename T, typename W, int D, int E, bool INTER, bool NORM>
__global__ void __launch_bounds__(256) rope_fwd_kernel(RopeArgs a) {
  using R = Run<T, E>;
  using L = Lane<E, INTER>;
  constexpr int LANES = D / (2 * E), GROUPS = 256 / LANES, STEP = 2 * R::BYTES * 256;
  extern __shared__ __align__(16) uint8_t smem[];
  const int l = threadIdx.x % LANES;
  const long long token = (long long)blockIdx.x * GROUPS + threadIdx.x / LANES;
  const bool on = token < (long long)a.s.B * a.s.S;
  const int s = on ? (int)(token % a.s.S) : 0, b = on ? (int)(token / a.s.S) : 0;
  const int key = (int)blockIdx.y >= a.s.q_chunks;
  const int h0 = ((int)blockIdx.y - (key ? a.s.q_chunks : 0)) * a.s.chunk;
  const int heads = min((key ? a.s.Hkv : a.s.Hq) - h0, a.s.chunk);
  L lane(a, l);
  const RowView xv = key ? a.x[1] : a.x[0], yv = key ? a.y[1] : a.y[0];
  const T* x0 = static_cast<const T*>(xv.ptr) + b * xv.sb + s * xv.ss + h0 * xv.sh;
  T* y0 = static_cast<T*>(yv.ptr) + b * yv.sb + s * yv.ss + h0 * yv.sh;
  const uint32_t ring = tc::smem_u32(smem) + threadIdx.x * R::UNIT;
  int asked = 0;
  auto ask = [&](uint32_t slot) {   // a token past the end (which reads the first one's rows) is not written
    if (asked < heads) {
      R::copy(slot, x0 + lane.c0);
      R::copy(slot + STEP / 2, x0 + lane.c1);
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
    ++asked;
    x0 += xv.sh;
  };
#pragma unroll
  for (int i = 0; i < kAhead - 1; ++i) ask(ring + i * STEP);
  uint64_t w[E];
#pragma unroll
  for (int i = 0; i < E; ++i) w[i] = twice(1.f);
  if constexpr (NORM) {
    const W* wp = static_cast<const W*>(key ? a.w[1] : a.w[0]);
    Run<W, E> run;
    run.load(wp + lane.c0);
    run.values(w);
    run.load(wp + lane.c1);
    run.values(w + E / 2);
  }
  lane.angles(a, l, b, s);
  const Turn<E, INTER> turn(lane, w, std::false_type{});   // with the weights
  unsigned slot = 0;
  for (int h = 0; h < heads; ++h) {
    ask(ring + (slot + kAhead - 1) % kAhead * STEP);
    asm volatile("cp.async.wait_group %0;" ::"n"(kAhead - 1) : "memory");
    uint64_t x[E];
    {
      R in;
      in.fetch(ring + slot * STEP);
      in.values(x);
      in.fetch(ring + slot * STEP + STEP / 2);
      in.values(x + E / 2);
    }
    slot = (slot + 1) % kAhead;
    uint64_t r = twice(1.f);
    if constexpr (NORM) {
      uint64_t sq = tc::mul_f32x2(x[0], x[0]);
#pragma unroll
      for (int i = 1; i < E; ++i) sq = tc::fma_f32x2(x[i], x[i], sq);
      r = twice(rsqrtf(fmaf(group_sum<LANES>(both(sq)), 1.f / D, a.s.eps)));
    }
    if (lane.turns) {
      turn(x);
    } else if constexpr (NORM) {
#pragma unroll
      for (int i = 0; i < E; ++i) x[i] = tc::mul_f32x2(x[i], turn.a[i]);
    }
    if constexpr (NORM) {
#pragma unroll
      for (int i = 0; i < E; ++i) x[i] = tc::mul_f32x2(x[i], r);
    }
    if (on) {
      R out;
      out.store(y0 + lane.c0, x);
      out.store(y0 + lane.c1, x + E / 2);
    }
    y0 += yv.sh;
  }
}

// As the forward, with the gradient of the output in and that of the input out. A block adds up its
// rows' weight gradients in registers, then over its groups in shared memory, and writes one row of
// partial sums, which rope_dw_kernel adds in block order.
template <typename T, typename W, int D, int E, bool INTER, bool NORM>
__global__ void __launch_bounds__(256) rope_bwd_kernel(RopeArgs a) {
  using R = Run<T, E>;
  using L = Lane<E, INTER>;
  constexpr int LANES = D / (2 * E), GROUPS = 256 / LANES, STEP = (NORM ? 4 : 2) * R::BYTES * 256, RUN = R::BYTES * 256;
  extern __shared__ __align__(16) uint8_t smem[];
  const int l = threadIdx.x % LANES, group = threadIdx.x / LANES;
  const long long token = (long long)blockIdx.x * GROUPS + group;
  const bool on = token < (long long)a.s.B * a.s.S;
  const int s = on ? (int)(token % a.s.S) : 0, b = on ? (int)(token / a.s.S) : 0;
  const int key = (int)blockIdx.y >= a.s.q_chunks;
  const int h0 = ((int)blockIdx.y - (key ? a.s.q_chunks : 0)) * a.s.chunk;
  const int heads = min((key ? a.s.Hkv : a.s.Hq) - h0, a.s.chunk);
  L lane(a, l);
  const RowView xv = key ? a.x[1] : a.x[0], yv = key ? a.y[1] : a.y[0], gv = key ? a.g[1] : a.g[0];
  const T* x0 = static_cast<const T*>(xv.ptr) + b * xv.sb + s * xv.ss + h0 * xv.sh;
  const T* g0 = static_cast<const T*>(gv.ptr) + b * gv.sb + s * gv.ss + h0 * gv.sh;
  T* y0 = static_cast<T*>(yv.ptr) + b * yv.sb + s * yv.ss + h0 * yv.sh;
  const uint32_t ring = tc::smem_u32(smem) + threadIdx.x * R::UNIT;
  int asked = 0;
  auto ask = [&](uint32_t slot) {
    if (asked < heads) {
      R::copy(slot, g0 + lane.c0);
      R::copy(slot + RUN, g0 + lane.c1);
      if constexpr (NORM) {
        R::copy(slot + 2 * RUN, x0 + lane.c0);
        R::copy(slot + 3 * RUN, x0 + lane.c1);
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
    ++asked;
    g0 += gv.sh;
    x0 += xv.sh;
  };
#pragma unroll
  for (int i = 0; i < kAhead - 1; ++i) ask(ring + i * STEP);
  uint64_t w[E], dw[E], one[E];
#pragma unroll
  for (int i = 0; i < E; ++i) {
    dw[i] = 0;
    one[i] = twice(1.f);
  }
  if constexpr (NORM) {
    const W* wp = static_cast<const W*>(key ? a.w[1] : a.w[0]);
    Run<W, E> run;
    run.load(wp + lane.c0);
    run.values(w);
    run.load(wp + lane.c1);
    run.values(w + E / 2);
  }
  lane.angles(a, l, b, s);
  const Turn<E, INTER> turn(lane, one, std::true_type{});
  unsigned slot = 0;
  for (int h = 0; h < heads; ++h) {
    ask(ring + (slot + kAhead - 1) % kAhead * STEP);
    asm volatile("cp.async.wait_group %0;" ::"n"(kAhead - 1) : "memory");
    const uint32_t at = ring + slot * STEP;
    slot = (slot + 1) % kAhead;
    R in;
    uint64_t g[E];
    in.fetch(at);
    in.values(g);
    in.fetch(at + RUN);
    in.values(g + E / 2);
    if (lane.turns) turn(g);
    if constexpr (NORM) {
      uint64_t x[E];
      in.fetch(at + 2 * RUN);
      in.values(x);
      in.fetch(at + 3 * RUN);
      in.values(x + E / 2);
      uint64_t t[E];
#pragma unroll
      for (int i = 0; i < E; ++i) t[i] = tc::mul_f32x2(g[i], w[i]);
      uint64_t sq2 = tc::mul_f32x2(x[0], x[0]), tx2 = tc::mul_f32x2(t[0], x[0]);
#pragma unroll
      for (int i = 1; i < E; ++i) {
        sq2 = tc::fma_f32x2(x[i], x[i], sq2);
        tx2 = tc::fma_f32x2(t[i], x[i], tx2);
      }
      const float sq = group_sum<LANES>(both(sq2)), tx = group_sum<LANES>(both(tx2));
      const float r = rsqrtf(fmaf(sq, 1.f / D, a.s.eps));
      const uint64_t r2 = twice(r), m2 = twice(-tx * (1.f / D) * r * r);
#pragma unroll
      for (int i = 0; i < E; ++i) {
        if (on) dw[i] = tc::fma_f32x2(g[i], tc::mul_f32x2(x[i], r2), dw[i]);
        g[i] = tc::mul_f32x2(r2, tc::fma_f32x2(x[i], m2, t[i]));
      }
    }
    if (on) {
      R out;
      out.store(y0 + lane.c0, g);
      out.store(y0 + lane.c1, g + E / 2);
    }
    y0 += yv.sh;
  }
  if constexpr (NORM) {
    let_next_kernel_start();
    __syncthreads();   // every lane is done with its slots
    float* part = reinterpret_cast<float*>(smem);   // [GROUPS][D]
#pragma unroll
    for (int i = 0; i < E; ++i) {
      float* at = part + group * D + (i < E / 2 ? lane.c0 + 2 * i : lane.c1 + 2 * i - E);
      tc::f32x2_split(dw[i], at[0], at[1]);
    }
    __syncthreads();
    for (int d = threadIdx.x; d < D; d += 256) {
      float sum = 0.f;
#pragma unroll 8
      for (int i = 0; i < GROUPS; ++i) sum += part[i * D + d];
      a.dw[((size_t)blockIdx.y * gridDim.x + blockIdx.x) * D + d] = sum;
    }
  }
}

// Adds the blocks' partial weight gradients in order, 16 features to a block: blockIdx.y 0 the queries' rows, 1 the keys'.
template <int D>
__global__ void __launch_bounds__(1024) rope_dw_kernel(const float* __restrict__ part, long long q_rows, long long rows,
                                                       float* __restrict__ dq_w, float* __restrict__ dk_w) {
  __shared__ float sums[64][17];
  wait_for_kernel_before();
  const long long first = blockIdx.y ? q_rows : 0, last = blockIdx.y ? rows : q_rows;
  const int f = threadIdx.x % 16, slice = threadIdx.x / 16, d = blockIdx.x * 16 + f;
  float sum = 0.f;
#pragma unroll 8
  for (long long i = first + slice; i < last; i += 64) sum += part[i * D + d];
  sums[slice][f] = sum;
  __syncthreads();
  if (slice != 0) return;
#pragma unroll 16
  for (int i = 1; i < 64; ++i) sum += sums[i][f];
  float* out = blockIdx.y ? dk_w : dq_w;
  if (out != nullptr) out[d] = sum;
}

// Heads a group of lanes takes, and the grid. More heads share a token's angles; fewer give more
// groups to spread over the SMs.
struct RopeGrid {
  int chunk, q_chunks, k_chunks;
  unsigned x;
};

// Features of a lane's runs. 8 make 16-byte copies of bf16 and half the work that a row costs besides its features (4 x 4096
// tokens of 40 heads: 54 us, 58 with 4; their backward at half the size 45 and 49), 4 take fewer angles and registers (one
// token of 8 sequences: 2.4 us, 3.1 with 8).
int run_of(const RopeShape& s, int dtype) {
  const bool many = (long long)s.B * s.S * (s.Hq + s.Hkv) >= 1LL << 17;
  return dtype == DT_BF16 && s.half % 8 == 0 && many ? 8 : 4;
}

RopeGrid rope_grid(const RopeShape& s, int D, int run) {
  const int groups = 256 / (D / (2 * run));
  const long long blocks = ((long long)s.B * s.S + groups - 1) / groups;
  const long long want = 2LL * sm_count();   // 8 and 1 measured slower where this decides (2042 tokens of 24 heads)
  RopeGrid g{32, 0, 0, 0};
  while (g.chunk > 1 && blocks * ((s.Hq + g.chunk - 1) / g.chunk + (s.Hkv + g.chunk - 1) / g.chunk) < want) g.chunk /= 2;
  g.q_chunks = (s.Hq + g.chunk - 1) / g.chunk;
  g.k_chunks = (s.Hkv + g.chunk - 1) / g.chunk;
  g.x = blocks > 0x7fffffffLL ? 0u : (unsigned)blocks;
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

template <auto KERNEL>
cudaError_t launch_rope(int smem, dim3 grid, const RopeArgs& a, cudaStream_t st) {
  static std::atomic<uint64_t> allowed{0};
  const cudaError_t e = allow_shared(KERNEL, smem, allowed);
  if (e != cudaSuccess) return e;
  KERNEL<<<grid, 256, smem, st>>>(a);
  count_launches(1);
  return cudaGetLastError();
}

template <typename F>
void by_type(const fa_rope_params* p, int run, F f) {
  auto by_pairs = [&](auto t, auto w, auto dim, auto e) {
    if (p->interleaved) f(t, w, dim, e, std::true_type{});
    else f(t, w, dim, e, std::false_type{});
  };
  auto by_run = [&](auto t, auto w, auto dim) {
    if constexpr (std::is_same_v<decltype(t), __nv_bfloat16>)
      if (run == 8) return by_pairs(t, w, dim, std::integral_constant<int, 8>{});
    by_pairs(t, w, dim, std::integral_constant<int, 4>{});
  };
  auto by_dim = [&](auto t, auto w) {
    if (p->D == 64) by_run(t, w, std::integral_constant<int, 64>{});
    else by_run(t, w, std::integral_constant<int, 128>{});
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
  if ((st = check_buffers(in, n, out, 2, side_by_side(q_out, p->Hq, k_out, p->Hkv, p->B, p->S, p->D, es))) != FA_OK) return st;
  if ((st = check_apart(out, 2, p, inv_freq, positions)) != FA_OK) return st;
  if (p->S == 0) return FA_OK;
  const int run = run_of(a.s, p->dtype);
  const RopeGrid g = rope_grid(a.s, p->D, run);
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
  cudaError_t e = cudaSuccess;
  by_type(p, run, [&](auto t, auto w, auto dim, auto e_run, auto inter) {
    using T = decltype(t);
    using W = decltype(w);
    constexpr int D = decltype(dim)::value, E = decltype(e_run)::value;
    constexpr bool INTER = decltype(inter)::value;
    if (p->norm) e = launch_rope<rope_fwd_kernel<T, W, D, E, INTER, true>>(ring_bytes<T, E>(1), grid, a, cs);
    else if constexpr (std::is_same_v<T, W>) e = launch_rope<rope_fwd_kernel<T, T, D, E, INTER, false>>(ring_bytes<T, E>(1), grid, a, cs);
  });
  return cuda_status(e, "norm and rotation launch");
}

size_t fa_qk_norm_rope_bwd_workspace_size(const fa_rope_params* p) {
  RopeShape s;
  if (check_rope(p, s) != FA_OK || !p->norm || p->S == 0) return 0;
  const RopeGrid g = rope_grid(s, p->D, run_of(s, p->dtype));
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
  // of a side without heads: zeros, where it is given
  out[2] = {dq_weight, p->norm && (p->Hq || dq_weight) ? (size_t)p->D * 4 : 0, "dq_weight"};
  out[3] = {dk_weight, p->norm && (p->Hkv || dk_weight) ? (size_t)p->D * 4 : 0, "dk_weight"};
  int n = 4;
  if ((st = check_small(p, q_weight, k_weight, inv_freq, positions, in, n)) != FA_OK) return st;
  if ((st = check_buffers(in, n, out, 4, side_by_side(dq, p->Hq, dk, p->Hkv, p->B, p->S, p->D, es))) != FA_OK) return st;
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
  const int run = run_of(a.s, p->dtype);
  const RopeGrid g = rope_grid(a.s, p->D, run);
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
  cudaError_t e = cudaSuccess;
  by_type(p, run, [&](auto t, auto w, auto dim, auto e_run, auto inter) {
    using T = decltype(t);
    using W = decltype(w);
    constexpr int D = decltype(dim)::value, E = decltype(e_run)::value;
    constexpr bool INTER = decltype(inter)::value;
    // the ring, which holds the groups' weight gradients at the end: 2 E x 256 floats
    constexpr int norm = ring_bytes<T, E>(2) > 2 * E * 256 * 4 ? ring_bytes<T, E>(2) : 2 * E * 256 * 4;
    if (p->norm) e = launch_rope<rope_bwd_kernel<T, W, D, E, INTER, true>>(norm, grid, a, cs);
    else if constexpr (std::is_same_v<T, W>) e = launch_rope<rope_bwd_kernel<T, T, D, E, INTER, false>>(ring_bytes<T, E>(1), grid, a, cs);
  });
  if (e == cudaSuccess && p->norm) {
    const long long q_rows = (long long)g.x * g.q_chunks, rows = q_rows + (long long)g.x * g.k_chunks;
    auto dw = p->D == 64 ? rope_dw_kernel<64> : rope_dw_kernel<128>;
    e = launch_after(dw, dim3(p->D / 16, 2), 1024, cs, a.dw, q_rows, rows, dq_weight, dk_weight);
    count_launches(1);
  }
  return cuda_status(e, "norm and rotation backward launch");
}

}  // extern "C"
