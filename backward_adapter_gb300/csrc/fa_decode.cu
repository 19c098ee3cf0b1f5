// Attention of the newest tokens of every sequence over its quantized cache, read in place
// (fa_decode): the serving form of the op, one to a few tokens per sequence.
//
// Mathematics. With G = Hq / Hkv query heads on a key/value head, the R = G * Sq query rows of one
// head all read the same keys. A block of 32 features of a key is d * n with whole numbers n, so
//     s_j = scale * sum_blocks d_jb <n_jb, q_b>,   o = sum_j sum_blocks (p_j d_jb) n_jb :
// the tensor cores multiply the whole numbers, exact in bf16, by q and by p * d, and the scales
// never touch the 8- or 4-bit data. Scores, softmax statistics and sums are fp32; p * d is rounded
// to bf16 for the second product (off by 2^-9 at most, as every key's weight on the training path).
//
// What bounds it: the planes are read once, 144 bytes a key for D = 128 in 4 bits, so HBM; next to
// that the instructions that turn packed bits into operands. Keys are the 16 rows of an
// mma.sync m16n8k16 and query rows its 8 columns: with 4 query rows a head a tcgen05 tile of 128
// rows would be 3% full, and its operands would have to be written to shared memory as bf16 first,
// four times the bytes that are read.
//
// A 4-bit number b becomes a bf16 by two instructions for two of them: its bits are put below the
// leading one of 16.0, which makes 16 + b. For K the difference to b - 8 is a multiple of the sum of
// a block's q, the products' starting value; for V it is subtracted (an exact bf16 operation),
// since there the difference would be far larger than what is summed.
//
// Every warp walks its own tiles of 32 keys through its own ring of shared memory (cp.async, no
// block barriers), with its own running maximum; a block's warps are joined in shared memory, and
// the blocks of a sequence, each a fixed number of keys, by a second kernel.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cmath>
#include <type_traits>

#include "fa_check.h"
#include "fa_device.cuh"
#include "kv_q8.cuh"
#include "tc_ptx.cuh"

namespace fa {
namespace {

constexpr int kMaxTokens = 16;
constexpr int kWarps = 4;
constexpr int kTile = 32;   // keys a warp takes at a time

struct DecodeArgs {
  CacheView c;
  const __nv_bfloat16* q;
  __nv_bfloat16* o;
  float* lse;
  const int64_t* lengths;
  float* part_o;         // [B, Hq, Sq, splits, D]: unnormalised, relative to part_ml's maximum
  float2* part_ml;       // [B, Hq, Sq, splits]: maximum (of scores in base 2) and sum
  unsigned* status;
  float scale2;          // scale * log2(e)
  int Hq, Sq, window, layout;
  int G, R;              // query heads and rows of a key/value head
  int span;              // keys of a block
  int splits;            // blocks of a (sequence, head)
};

// The keys a sequence's queries may see: [lo, len), lo on a tile's border.
struct Range { int len, lo; };

__device__ __forceinline__ Range key_range(const DecodeArgs& a, int b, bool report) {
  long long n = a.lengths != nullptr ? __ldg(a.lengths + b) : a.c.S;
  if (n < 0 || n > a.c.S) {
    if (report && a.status != nullptr) atomicCAS(a.status, 0u, 0x40000000u | kSiteDecodeLength);
    n = n < 0 ? 0 : a.c.S;
  }
  Range r{(int)n, 0};
  if (a.window > 0) {
    const long long lo = n - a.Sq - a.window;   // the first token's furthest key
    r.lo = lo > 0 ? (int)lo & ~(kTile - 1) : 0;
  }
  return r;
}

// Element offset of query row r (head r / Sq of the group, token r % Sq) in q and o.
__device__ __forceinline__ size_t q_offset(const DecodeArgs& a, int b, int h, int r) {
  const int head = h * a.G + r / a.Sq, i = r % a.Sq;
  return (a.layout ? ((size_t)b * a.Sq + i) * a.Hq + head : ((size_t)b * a.Hq + head) * a.Sq + i) * a.c.D;
}

__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool on) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(on ? 16 : 0) : "memory");
}
template <int N>
__device__ __forceinline__ void cp_async_small(uint32_t dst, const void* src, bool on) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(dst), "l"(src), "n"(N), "r"(on ? N : 0) : "memory");
}

__device__ __forceinline__ uint32_t lds32(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared.b32 %0, [%1];" : "=r"(v) : "r"(a));
  return v;
}
__device__ __forceinline__ uint2 lds64(uint32_t a) {
  uint2 v;
  asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a));
  return v;
}

__device__ __forceinline__ void mma(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                    uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

// Four-bit numbers of both halves of x at bit `at`, as the bf16 pair 16 + b.
template <int AT>
__device__ __forceinline__ uint32_t nibbles(uint32_t x) {
  const uint32_t y = AT < 3 ? x << (3 - AT) : x >> (AT - 3);
  return (y & 0x00780078u) | 0x41804180u;
}
__device__ __forceinline__ uint32_t minus24(uint32_t x) {
  const __nv_bfloat162 k = __halves2bfloat162(__ushort_as_bfloat16(0x41C0), __ushort_as_bfloat16(0x41C0));
  const __nv_bfloat162 r = __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&x), k);
  return *reinterpret_cast<const uint32_t*>(&r);
}

// Where things are in a ring slot, and how a row's 16-byte pieces are permuted there so that the
// fragments' loads meet no bank twice.
template <int D, bool Q4>
struct Slot {
  static constexpr int ROW = Q4 ? D / 2 : D;      // bytes of a key's numbers
  static constexpr int PIECES = ROW / 16;
  static constexpr int NB = D / 32;               // blocks
  static constexpr int SC = NB * 2;               // bytes of a key's scales
  static constexpr int V_OFF = kTile * ROW;
  static constexpr int KD_OFF = 2 * kTile * ROW;
  static constexpr int VD_OFF = KD_OFF + kTile * SC;
  static constexpr int BYTES = VD_OFF + kTile * SC;
  static constexpr int STAGES = BYTES <= 5120 ? 3 : 2;
  __device__ static __forceinline__ int piece(int row, int p) {
    constexpr int PER = 128 / ROW;                // rows in 128 bytes
    return p ^ ((row / PER) & (PIECES - 1));
  }
};

template <int NB>
__device__ __forceinline__ void load_scales(uint32_t at, float (&d)[NB]) {
  if constexpr (NB == 4) {
    const uint2 u = lds64(at);
    const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&u.x));
    const float2 b = __half22float2(*reinterpret_cast<const __half2*>(&u.y));
    d[0] = a.x; d[1] = a.y; d[2] = b.x; d[3] = b.y;
  } else {
    const uint32_t u = lds32(at);
    const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&u));
    d[0] = a.x; d[1] = a.y;
  }
}

// One block: `span` keys of one (sequence, key/value head), for NT * 8 of its query rows.
template <int D, bool Q4, int NT>
__global__ void __launch_bounds__(kWarps * 32) decode_kernel(DecodeArgs a) {
  using S = Slot<D, Q4>;
  constexpr int NB = S::NB;
  extern __shared__ __align__(128) uint8_t smem[];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int g = lane >> 2, t = lane & 3;
  const int split = blockIdx.x % a.splits, head = blockIdx.x / a.splits;   // head: of all sequences
  const int b = head / a.c.Hkv, h = head % a.c.Hkv;
  const int r0 = blockIdx.y * NT * 8;
  const Range kr = key_range(a, b, split == 0 && h == 0 && r0 == 0 && threadIdx.x == 0);
  const int k0 = kr.lo + split * a.span;
  if (k0 >= kr.len && a.splits > 1) return;       // the joining kernel knows
  const int k1 = min(kr.len, k0 + a.span);
  const int tiles = k0 < k1 ? (k1 - k0 + kTile - 1) / kTile : 0;
  const size_t plane = (size_t)head * a.c.S;

  const uint32_t ring = tc::smem_u32(smem) + warp * (S::STAGES * S::BYTES);
  auto load = [&](int tile, int slot) {
    const int first = k0 + tile * kTile;
    const uint32_t at = ring + slot * S::BYTES;
#pragma unroll
    for (int i = 0; i < S::PIECES; ++i) {
      const int c = lane + 32 * i, row = c / S::PIECES, p = c % S::PIECES;
      const bool on = first + row < k1;
      const size_t src = (plane + (on ? first + row : 0)) * S::ROW + 16 * p;
      const uint32_t dst = at + row * S::ROW + 16 * S::piece(row, p);
      cp_async16(dst, static_cast<const uint8_t*>(a.c.k_q) + src, on);
      cp_async16(dst + S::V_OFF, static_cast<const uint8_t*>(a.c.v_q) + src, on);
    }
    const bool on = first + lane < k1;
    const size_t src = (plane + (on ? first + lane : 0)) * NB;
    cp_async_small<S::SC>(at + S::KD_OFF + lane * S::SC, a.c.k_d + src, on);
    cp_async_small<S::SC>(at + S::VD_OFF + lane * S::SC, a.c.v_d + src, on);
  };
  auto commit = [] { asm volatile("cp.async.commit_group;" ::: "memory"); };

#pragma unroll
  for (int i = 0; i < S::STAGES - 1; ++i) {
    if (warp + i * kWarps < tiles) load(warp + i * kWarps, i);
    commit();
  }

  // the query rows as operands: lane (g, t) holds, of row g, the features that its part of a key's
  // block holds
  uint32_t qf[NT][NB][2][2];
  float bias[NT][NB][2];   // -24 * (sum of a block's q) of columns 2 t and 2 t + 1
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    const int r = r0 + n * 8 + g;
    const __nv_bfloat16* src = a.q + (r < a.R ? q_offset(a, b, h, r) : 0);
#pragma unroll
    for (int k = 0; k < NB; ++k) {
      float sum = 0.f;
#pragma unroll
      for (int st = 0; st < 2; ++st)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const int f0 = 32 * k + (Q4 ? 16 * st + 4 * t + j : 8 * t + 4 * st + 2 * j), f1 = f0 + (Q4 ? 2 : 1);
          uint32_t v = 0;
          if (r < a.R) v = (uint32_t)__bfloat16_as_ushort(src[f0]) | ((uint32_t)__bfloat16_as_ushort(src[f1]) << 16);
          qf[n][k][st][j] = v;
          sum += __uint_as_float(v << 16) + __uint_as_float(v & 0xffff0000u);
        }
      sum += __shfl_xor_sync(0xffffffffu, sum, 1);
      sum += __shfl_xor_sync(0xffffffffu, sum, 2);
      bias[n][k][0] = Q4 ? -24.f * __shfl_sync(0xffffffffu, sum, 8 * t) : 0.f;
      bias[n][k][1] = Q4 ? -24.f * __shfl_sync(0xffffffffu, sum, 8 * t + 4) : 0.f;
    }
  }

  float acc[NT][2 * NB][4];   // rows: features of block k, half-tile m; columns: query rows 2 t, 2 t + 1
  float mx[NT][2], sum[NT][2];
#pragma unroll
  for (int n = 0; n < NT; ++n) {
#pragma unroll
    for (int i = 0; i < 2 * NB; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) acc[n][i][j] = 0.f;
    mx[n][0] = mx[n][1] = -CUDART_INF_F;
    sum[n][0] = sum[n][1] = 0.f;
  }
  // a tile is on an edge when some query row does not see all of it
  const int all_to = kr.len - a.Sq, all_from = a.window > 0 ? kr.len - 1 - a.window : 0;

  int slot = 0;
  for (int tile = warp; tile < tiles; tile += kWarps) {
    {
      const int next = tile + (S::STAGES - 1) * kWarps;
      if (next < tiles) load(next, slot == 0 ? S::STAGES - 1 : slot - 1);
      commit();
    }
    asm volatile("cp.async.wait_group %0;" ::"n"(S::STAGES - 1) : "memory");
    __syncwarp();
    const uint32_t at = ring + slot * S::BYTES;
    const int first = k0 + tile * kTile;
    const bool edge = first + kTile - 1 > all_to || first < all_from;

    // scores of 2 x 16 keys
    float s[NT][2][4];
#pragma unroll
    for (int m = 0; m < 2; ++m) {
      float d0[NB], d1[NB];
      load_scales<NB>(at + S::KD_OFF + (16 * m + g) * S::SC, d0);
      load_scales<NB>(at + S::KD_OFF + (16 * m + g + 8) * S::SC, d1);
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int j = 0; j < 4; ++j) s[n][m][j] = 0.f;
#pragma unroll
      for (int k = 0; k < NB; ++k) {
        uint32_t f[2][4];   // [row g or g + 8][two k-steps of two registers]
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const int row = 16 * m + g + 8 * u;
          if constexpr (Q4) {
            const uint32_t w = lds32(at + row * S::ROW + 16 * S::piece(row, k) + 4 * t);
            f[u][0] = nibbles<0>(w);
            f[u][1] = nibbles<8>(w);
            f[u][2] = nibbles<4>(w);
            f[u][3] = nibbles<12>(w);
          } else {
            const uint2 w = lds64(at + row * S::ROW + 16 * S::piece(row, 2 * k + (t >> 1)) + 8 * (t & 1));
            const uint32_t x = w.x ^ 0x80808080u, y = w.y ^ 0x80808080u;
            f[u][0] = tc::pack_bf16x2(s8_to_f32(x, 0), s8_to_f32(x, 1));
            f[u][1] = tc::pack_bf16x2(s8_to_f32(x, 2), s8_to_f32(x, 3));
            f[u][2] = tc::pack_bf16x2(s8_to_f32(y, 0), s8_to_f32(y, 1));
            f[u][3] = tc::pack_bf16x2(s8_to_f32(y, 2), s8_to_f32(y, 3));
          }
        }
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          float c[4] = {bias[n][k][0], bias[n][k][1], bias[n][k][0], bias[n][k][1]};
          mma(c, f[0][0], f[1][0], f[0][1], f[1][1], qf[n][k][0][0], qf[n][k][0][1]);
          mma(c, f[0][2], f[1][2], f[0][3], f[1][3], qf[n][k][1][0], qf[n][k][1][1]);
          s[n][m][0] = fmaf(d0[k], c[0], s[n][m][0]);
          s[n][m][1] = fmaf(d0[k], c[1], s[n][m][1]);
          s[n][m][2] = fmaf(d1[k], c[2], s[n][m][2]);
          s[n][m][3] = fmaf(d1[k], c[3], s[n][m][3]);
        }
      }
    }

    // softmax weights, relative to the running maximum of each column
    uint32_t hidden[NT];   // bit 4 m + j: pair j of half m
#pragma unroll
    for (int n = 0; n < NT; ++n) {
#pragma unroll
      for (int m = 0; m < 2; ++m)
#pragma unroll
        for (int j = 0; j < 4; ++j) s[n][m][j] *= a.scale2;
      hidden[n] = 0;
      if (edge) {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const int pos = kr.len - a.Sq + (r0 + n * 8 + 2 * t + j) % a.Sq;
#pragma unroll
          for (int m = 0; m < 2; ++m)
#pragma unroll
            for (int u = 0; u < 2; ++u) {
              const int key = first + 16 * m + g + 8 * u;
              if (key > pos || (a.window > 0 && pos - key > a.window)) {
                s[n][m][2 * u + j] = -CUDART_INF_F;
                hidden[n] |= 1u << (4 * m + 2 * u + j);
              }
            }
        }
      }
      float top[2];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        top[j] = fmaxf(fmaxf(s[n][0][j], s[n][0][j + 2]), fmaxf(s[n][1][j], s[n][1][j + 2]));
        top[j] = fmaxf(top[j], __shfl_xor_sync(0xffffffffu, top[j], 4));
        top[j] = fmaxf(top[j], __shfl_xor_sync(0xffffffffu, top[j], 8));
        top[j] = fmaxf(top[j], __shfl_xor_sync(0xffffffffu, top[j], 16));
      }
      const bool up = top[0] > mx[n][0] || top[1] > mx[n][1];
      if (__any_sync(0xffffffffu, up)) {
        float f[2];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const float now = fmaxf(mx[n][j], top[j]);
          f[j] = now > mx[n][j] ? exp2_fast(mx[n][j] - now) : 1.f;   // 0 from a maximum of -inf
          mx[n][j] = now;
          sum[n][j] *= f[j];
        }
#pragma unroll
        for (int i = 0; i < 2 * NB; ++i) {
          acc[n][i][0] *= f[0];
          acc[n][i][1] *= f[1];
          acc[n][i][2] *= f[0];
          acc[n][i][3] *= f[1];
        }
      }
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const float base = mx[n][j] == -CUDART_INF_F ? 0.f : mx[n][j];   // nothing seen so far: all weights 0
#pragma unroll
        for (int m = 0; m < 2; ++m)
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            const float p = exp2_fast(s[n][m][2 * u + j] - base);
            s[n][m][2 * u + j] = p;
            sum[n][j] += p;
          }
      }
    }

    // o += V^T (p d)
#pragma unroll
    for (int m = 0; m < 2; ++m) {
      float d0[NB], d1[NB];
      load_scales<NB>(at + S::VD_OFF + (16 * m + g) * S::SC, d0);
      load_scales<NB>(at + S::VD_OFF + (16 * m + g + 8) * S::SC, d1);
#pragma unroll
      for (int k = 0; k < NB; ++k) {
        uint32_t f[2][4];   // [keys 2 t, 2 t + 1 or those + 8][features]
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const int row = 16 * m + 8 * u + 2 * t;
          if constexpr (Q4) {
            // bytes 2 g, 2 g + 1 of the block, of two keys
            const uint32_t wa = lds32(at + S::V_OFF + row * S::ROW + 16 * S::piece(row, k) + 4 * (g >> 1));
            const uint32_t wb = lds32(at + S::V_OFF + (row + 1) * S::ROW + 16 * S::piece(row + 1, k) + 4 * (g >> 1));
            const uint32_t x = __byte_perm(wa, wb, (g & 1) ? 0x7632u : 0x5410u);
            f[u][0] = minus24(nibbles<0>(x));    // feature 2 g
            f[u][1] = minus24(nibbles<8>(x));    // 2 g + 1
            f[u][2] = minus24(nibbles<4>(x));    // 16 + 2 g
            f[u][3] = minus24(nibbles<12>(x));   // 17 + 2 g
          } else {
            const int p = 2 * k + (g >> 2);
            const uint32_t x = lds32(at + S::V_OFF + row * S::ROW + 16 * S::piece(row, p) + 4 * (g & 3)) ^ 0x80808080u;
            const uint32_t y =
                lds32(at + S::V_OFF + (row + 1) * S::ROW + 16 * S::piece(row + 1, p) + 4 * (g & 3)) ^ 0x80808080u;
#pragma unroll
            for (int i = 0; i < 4; ++i) f[u][i] = tc::pack_bf16x2(s8_to_f32(x, i), s8_to_f32(y, i));   // 4 g + i
          }
        }
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          float w[4] = {s[n][m][0] * d0[k], s[n][m][1] * d0[k], s[n][m][2] * d1[k], s[n][m][3] * d1[k]};
          if (edge) {   // a hidden key's scale may be anything
#pragma unroll
            for (int j = 0; j < 4; ++j) w[j] = (hidden[n] >> (4 * m + j)) & 1u ? 0.f : w[j];
          }
          const uint32_t b0 = transpose8x8(tc::pack_bf16x2(w[0], w[1]));
          const uint32_t b1 = transpose8x8(tc::pack_bf16x2(w[2], w[3]));
          mma(acc[n][2 * k], f[0][0], f[0][1], f[1][0], f[1][1], b0, b1);
          mma(acc[n][2 * k + 1], f[0][2], f[0][3], f[1][2], f[1][3], b0, b1);
        }
      }
    }
    __syncwarp();   // the slot is read: the next load into it may begin
    slot = slot == S::STAGES - 1 ? 0 : slot + 1;
  }
  asm volatile("cp.async.wait_all;" ::: "memory");

  // join the block's warps: [warp][query row][D], and their maxima and sums
  __syncthreads();
  float* so = reinterpret_cast<float*>(smem);
  float2* sml = reinterpret_cast<float2*>(smem + kWarps * NT * 8 * D * 4);
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      float l = sum[n][j];
      l += __shfl_xor_sync(0xffffffffu, l, 4);
      l += __shfl_xor_sync(0xffffffffu, l, 8);
      l += __shfl_xor_sync(0xffffffffu, l, 16);
      const int col = n * 8 + 2 * t + j;
      if (g == 0) sml[warp * NT * 8 + col] = make_float2(mx[n][j], l);
      float* row = so + ((size_t)warp * NT * 8 + col) * D;
#pragma unroll
      for (int i = 0; i < 2 * NB; ++i) {
        const int f = 32 * (i / 2) + (Q4 ? 16 * (i % 2) + 2 * g : 4 * g + 2 * (i % 2));
        *reinterpret_cast<float2*>(row + f) = make_float2(acc[n][i][j], acc[n][i][j + 2]);
      }
    }
  __syncthreads();
  constexpr int PER = D / 4;   // threads of a row
  for (int i = threadIdx.x; i < NT * 8 * PER; i += kWarps * 32) {
    const int col = i / PER, f = i % PER * 4, r = r0 + col;
    if (r >= a.R) continue;
    float top = -CUDART_INF_F;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) top = fmaxf(top, sml[w * NT * 8 + col].x);
    float l = 0.f;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const float2 ml = sml[w * NT * 8 + col];
      const float k = ml.x == -CUDART_INF_F ? 0.f : exp2_fast(ml.x - top);
      const float4 x = *reinterpret_cast<const float4*>(so + ((size_t)w * NT * 8 + col) * D + f);
      l = fmaf(k, ml.y, l);
      o.x = fmaf(k, x.x, o.x);
      o.y = fmaf(k, x.y, o.y);
      o.z = fmaf(k, x.z, o.z);
      o.w = fmaf(k, x.w, o.w);
    }
    const size_t row = ((size_t)b * a.Hq + h * a.G) * a.Sq + r;   // of lse and the partials
    if (a.splits > 1) {
      const size_t at = row * a.splits + split;
      *reinterpret_cast<float4*>(a.part_o + at * D + f) = o;
      if (f == 0) a.part_ml[at] = make_float2(top, l);
    } else {
      const float inv = l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l);
      uint2 u = make_uint2(tc::pack_bf16x2(o.x * inv, o.y * inv), tc::pack_bf16x2(o.z * inv, o.w * inv));
      *reinterpret_cast<uint2*>(a.o + q_offset(a, b, h, r) + f) = u;
      if (f == 0) a.lse[row] = l == 0.f ? 0.f : (top + log2f(l)) * 0.6931471805599453f;
    }
  }
}

// Joins the blocks of one query row: 8 warps take its blocks in turn, four features a lane (D = 128)
// or two (D = 64), and are joined in order.
template <int D>
__global__ void __launch_bounds__(256) decode_join_kernel(DecodeArgs a) {
  constexpr int F = D / 32;
  __shared__ float so[8][D];
  __shared__ float2 sml[8];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const long long row = blockIdx.x;
  const int i = (int)(row % a.Sq), head = (int)(row / a.Sq % a.Hq), b = (int)(row / a.Sq / a.Hq);
  const Range kr = key_range(a, b, false);
  const int n = kr.len > kr.lo ? (kr.len - kr.lo + a.span - 1) / a.span : 0;
  float top = -CUDART_INF_F, l = 0.f, o[F];
#pragma unroll
  for (int j = 0; j < F; ++j) o[j] = 0.f;
  for (int s = warp; s < n; s += 8) {
    const size_t at = (size_t)row * a.splits + s;
    const float2 ml = a.part_ml[at];
    if (ml.x == -CUDART_INF_F && ml.y == 0.f) continue;   // saw nothing (a sum that is not a number stays one)
    const float now = fmaxf(top, ml.x), k0 = exp2_fast(top - now), k1 = exp2_fast(ml.x - now);
    top = now;
    l = l * k0 + ml.y * k1;
#pragma unroll
    for (int j = 0; j < F; ++j) o[j] = o[j] * k0 + a.part_o[at * D + lane * F + j] * k1;
  }
  if (lane == 0) sml[warp] = make_float2(top, l);
#pragma unroll
  for (int j = 0; j < F; ++j) so[warp][lane * F + j] = o[j];
  __syncthreads();
  if (threadIdx.x >= D) return;
  top = -CUDART_INF_F;
  for (int w = 0; w < 8; ++w) top = fmaxf(top, sml[w].x);
  l = 0.f;
  float x = 0.f;
  for (int w = 0; w < 8; ++w) {
    if (sml[w].x == -CUDART_INF_F && sml[w].y == 0.f) continue;
    const float k = exp2_fast(sml[w].x - top);
    l = fmaf(k, sml[w].y, l);
    x = fmaf(k, so[w][threadIdx.x], x);
  }
  const size_t at = (a.layout ? ((size_t)b * a.Sq + i) * a.Hq + head : (size_t)row) * D;
  a.o[at + threadIdx.x] = __float2bfloat16_rn(l == 0.f ? 0.f : x / l);
  if (threadIdx.x == 0) a.lse[row] = l == 0.f ? 0.f : (top + log2f(l)) * 0.6931471805599453f;
}

struct DecodePlan {
  int nt, span, splits, row_blocks;
  size_t ml_off, total;
};

DecodePlan plan_decode(const fa_decode_params* p, const CacheView& c) {
  DecodePlan d{};
  const int R = p->Hq / c.Hkv * p->Sq;
  d.nt = R <= 8 ? 1 : 2;
  d.row_blocks = (R + 8 * d.nt - 1) / (8 * d.nt);
  const long long most = p->window > 0 && p->window < c.S ? (long long)p->window + p->Sq + kTile - 1 : c.S;
  const int keys = (int)(most < c.S ? most : c.S);
  const long long heads = (long long)c.B * c.Hkv * d.row_blocks;
  // keys of a block: enough blocks for several on every SM, down to two tiles a warp
  d.span = 1024;
  while (d.span > 2 * kWarps * kTile && heads * ((keys + d.span - 1) / d.span) < 6LL * sm_count()) d.span /= 2;
  if (keys <= 512) d.span = 512;   // one block, and no joining kernel
  d.splits = (keys + d.span - 1) / d.span;
  if (d.splits > 1) {
    const size_t rows = (size_t)c.B * p->Hq * p->Sq * d.splits;
    d.ml_off = align_up(rows * c.D * 4);
    d.total = d.ml_off + align_up(rows * 8);
  }
  return d;
}

fa_status check_decode(const fa_decode_params* p, const fa_cache* c, CacheView& cv) {
  clear_error();
  if (p == nullptr) { set_error("params is NULL"); return FA_ERR_INVALID_ARG; }
  const fa_status st = check_cache(c, cv);
  if (st != FA_OK) return st;
  if (p->Hq < 1 || p->Hq > 65535) { set_error("Hq=%d outside [1, 65535]", p->Hq); return FA_ERR_INVALID_ARG; }
  if (p->Hq % cv.Hkv != 0) { set_error("Hq=%d is not a multiple of Hkv=%d", p->Hq, cv.Hkv); return FA_ERR_INVALID_ARG; }
  if (p->Sq < 0 || p->Sq > kMaxTokens) { set_error("Sq=%d outside [0, %d]", p->Sq, kMaxTokens); return FA_ERR_INVALID_ARG; }
  if (p->window < 0) { set_error("window=%d must be >= 0 (0 = no window)", p->window); return FA_ERR_INVALID_ARG; }
  if (p->layout != FA_LAYOUT_BHSD && p->layout != FA_LAYOUT_BSHD) { set_error("layout=%d invalid", p->layout); return FA_ERR_INVALID_ARG; }
  if (!std::isfinite(p->scale)) { set_error("scale is not finite"); return FA_ERR_INVALID_ARG; }
  if (p->reserved != 0) { set_error("reserved field must be 0"); return FA_ERR_INVALID_ARG; }
  return FA_OK;
}

template <int D, bool Q4, int NT>
cudaError_t launch_decode(const DecodeArgs& a, dim3 grid, cudaStream_t st) {
  using S = Slot<D, Q4>;
  constexpr int ring = kWarps * S::STAGES * S::BYTES, join = kWarps * NT * 8 * (D * 4 + 8);
  constexpr int bytes = ring > join ? ring : join;
  cudaError_t e = cudaFuncSetAttribute(decode_kernel<D, Q4, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e != cudaSuccess) return e;
  decode_kernel<D, Q4, NT><<<grid, kWarps * 32, bytes, st>>>(a);
  count_launches(1);
  return cudaGetLastError();
}

}  // namespace
}  // namespace fa

using namespace fa;

extern "C" {

size_t fa_decode_workspace_size(const fa_decode_params* p, const fa_cache* c) {
  CacheView cv;
  if (check_decode(p, c, cv) != FA_OK || p->Sq == 0) return 0;
  return plan_decode(p, cv).total;
}

fa_status fa_decode(const fa_decode_params* p, const void* q, const fa_cache* c, const int64_t* lengths, void* o,
                    float* lse, void* ws, size_t ws_bytes, void* stream) {
  CacheView cv;
  fa_status st = check_decode(p, c, cv);
  if (st != FA_OK) return st;
  const size_t rows = (size_t)cv.B * p->Hq * p->Sq;
  Span all[8];
  cache_spans(cv, all);
  all[4] = {q, rows * cv.D * 2, "q"};
  Span* out = all + 5;
  out[0] = {o, rows * cv.D * 2, "o"};
  out[1] = {lse, rows * 4, "lse"};
  all[7] = {lengths, lengths != nullptr ? (size_t)cv.B * 8 : 0, "lengths"};
  if ((st = check_buffers(all, 5, out, 2)) != FA_OK) return st;
  if ((uintptr_t)lengths % 8 != 0) { set_error("lengths must be 8-byte aligned"); return FA_ERR_INVALID_ARG; }
  for (int i = 0; i < 2; ++i)
    if (overlaps(out[i], all[7])) { set_error("output %s overlaps input lengths", out[i].name); return FA_ERR_INVALID_ARG; }
  if (p->Sq == 0) return FA_OK;
  const DecodePlan plan = plan_decode(p, cv);
  if ((st = check_ws(ws, ws_bytes, plan.total, all, 8)) != FA_OK) return st;
  DecodeArgs a{};
  a.c = cv;
  a.q = static_cast<const __nv_bfloat16*>(q);
  a.o = static_cast<__nv_bfloat16*>(o);
  a.lse = lse;
  a.lengths = lengths;
  a.part_o = static_cast<float*>(ws);
  a.part_ml = plan.splits > 1 ? reinterpret_cast<float2*>(static_cast<char*>(ws) + plan.ml_off) : nullptr;
  a.status = device_status_ptr();
  a.scale2 = p->scale * 1.4426950408889634f;
  a.Hq = p->Hq;
  a.Sq = p->Sq;
  a.window = p->window;
  a.layout = p->layout;
  a.G = p->Hq / cv.Hkv;
  a.R = a.G * p->Sq;
  a.span = plan.span;
  a.splits = plan.splits;
  const long long blocks = (long long)cv.B * cv.Hkv * plan.splits;
  if (plan.row_blocks > 65535 || blocks > 0x7fffffffLL || rows > 0x7fffffffULL) { set_error("too many query rows for one launch"); return FA_ERR_UNSUPPORTED; }
  const dim3 grid((unsigned)blocks, (unsigned)plan.row_blocks);
  cudaStream_t cs = (cudaStream_t)stream;
  auto go = [&](auto dim, auto q4) {
    constexpr int D = decltype(dim)::value;
    constexpr bool Q4 = decltype(q4)::value;
    return plan.nt == 1 ? launch_decode<D, Q4, 1>(a, grid, cs) : launch_decode<D, Q4, 2>(a, grid, cs);
  };
  using D64 = std::integral_constant<int, 64>;
  using D128 = std::integral_constant<int, 128>;
  cudaError_t e;
  if (cv.q4) e = cv.D == 64 ? go(D64{}, std::true_type{}) : go(D128{}, std::true_type{});
  else e = cv.D == 64 ? go(D64{}, std::false_type{}) : go(D128{}, std::false_type{});
  if (e == cudaSuccess && plan.splits > 1) {
    if (cv.D == 64) decode_join_kernel<64><<<(unsigned)rows, 256, 0, cs>>>(a);
    else decode_join_kernel<128><<<(unsigned)rows, 256, 0, cs>>>(a);
    count_launches(1);
    e = cudaGetLastError();
  }
  return cuda_status(e, "decode launch");
}

}  // extern "C"
