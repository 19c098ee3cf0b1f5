// The attention weight that every key of a quantized cache got from a chunk of new tokens (fa_cache_weights), or from decoded ones
// (fa_cache_weights_decoded).
//
// Mathematics. P_ij = exp(scale <q_i, k_j> - lse_i) summed over the rows i (tokens and query heads of the key's head) that see
// key j. With K as the left operand the products S^T = K Q^T have a key for each lane of TMEM and a row for each column, so
// that a thread adds up a key's weights along its lane, in registers: no atomics, no second pass, a fixed order.
//
// Up to 16 rows (a step's tokens): the keys' bytes are what there is to read, 72 a key for D = 128 in 4 bits, and turning them
// into bf16 what there is to do. A warp has the keys of a chunk, 16 at a time as the rows of mma.sync m16n8k16, its lanes a
// quarter of a row each, from memory to operand without shared memory: which features a lane has in which step is its own
// choice, as long as it has the same ones of q. A tcgen05 tile would take the operands through shared memory and two barriers.
//
// More rows: a block has 256 keys at a time, two tiles of 128, made bf16 operands once (kv_tile.cuh), and all rows that see one
// of them go by, 128 at a time, which halves what the blocks read of Q from L2 against 128 keys. A block stays on its SM for all
// its keys: warps 1-7 bring the rows into a ring and make the operands of the next 256 keys in between, warp 0 issues the MMAs,
// and of warps 8-23 two threads own a key, each half of the rows; each tile's products are in two buffers.
//
// Measured (device time): a token of 64 sequences of 1024 to 8192 keys, 32 heads on 8, D = 128 in 4 bits: 85 us, 2.4 TB/s of K and
// weights, 36% of the measured copy rate (issue 60% busy, ALU 51%: turning bits into operands, with 20 warps an SM to wait for
// memory; by tcgen05 tiles 295). 512 tokens over 67,584 keys in 8 bits, 16 heads on 4: 184 us, 0.77 PFLOP/s. No unit bounds it: the
// products are 73 us (tensor cores 33% busy), its 551 million exponentials 57 at the measured 32 a cycle and SM (XU 36%), and issue is
// 64% busy; a copy without exponentials takes 129. It is the way of each tile of rows from L2 to operands, products, TMEM and sums.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cfloat>
#include <type_traits>

#include "fa_check.h"
#include "fa_device.cuh"
#include "kv_tile.cuh"
#include "tc_ptx.cuh"

namespace fa {
namespace {

using namespace tc;

constexpr float kLog2e = 1.4426950408889634f;
constexpr int kThreads = 768;
constexpr int kLoaders = 7;             // warps that bring rows and make operands
// Registers of a thread: what 768 are launched with, and what warps 0-7 and those that add make of it.
constexpr int kRegsLaunch = 80, kRegsLoad = 112, kRegsAdd = 64;
static_assert(2 * kRegsLoad + 4 * kRegsAdd <= 6 * kRegsLaunch, "register split exceeds the launch's");

struct WeightArgs {
  CacheView c;
  PageView pages;
  const __nv_bfloat16* q;
  const float* lse;
  const int64_t* lengths;
  const int64_t* count;
  const float* weights;
  float* out;
  unsigned* status;
  long long W;
  float sl2;         // scale log2(e)
  int Hq, Sq, window, layout, G;
};

// The sequence's keys and tokens, and a report of what is out of range.
__device__ __forceinline__ void read_lengths(const WeightArgs& a, int b, bool report, int& len, int& n) {
  const long long length = a.lengths != nullptr ? __ldg(a.lengths + b) : a.c.S;
  const long long tokens = a.count != nullptr ? __ldg(a.count + b) : a.Sq;
  len = (int)min(max(length, 0LL), (long long)a.c.S);
  n = (int)min(max(tokens, 0LL), (long long)a.Sq);
  if (report && (len != length || n != tokens || len > a.W) && a.status != nullptr) atomicCAS(a.status, 0u, 0x40000000u | kSiteDecodeLength);
}

__device__ __forceinline__ void mma_bf16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// A lane's quarter of rows g and g + 8 of a run of 16 keys, as it is stored.
template <int D, bool Q4>
struct Quarter {
  static constexpr int ROW = Q4 ? D / 2 : D, W = ROW / 16;   // bytes of a row, words of a quarter
  uint32_t w[2][W];
  uint16_t d[2];
  __device__ __forceinline__ void load(const WeightArgs& a, long long row, int keys) {
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int r = g + 8 * i;
#pragma unroll
      for (int j = 0; j < W; ++j) w[i][j] = Q4 ? 0x88888888u : 0u;
      d[i] = 0;
      if (row >= 0 && r < keys) {
        const uint8_t* src = static_cast<const uint8_t*>(a.c.k_q) + (row + r) * ROW + t * (ROW / 4);
        if constexpr (W == 2) {
          asm volatile("ld.global.nc.L1::no_allocate.v2.b32 {%0, %1}, [%2];" : "=r"(w[i][0]), "=r"(w[i][1]) : "l"(src));
        } else {
#pragma unroll
          for (int j = 0; j < W; j += 4)
            asm volatile("ld.global.nc.L1::no_allocate.v4.b32 {%0, %1, %2, %3}, [%4];"
                         : "=r"(w[i][j]), "=r"(w[i][j + 1]), "=r"(w[i][j + 2]), "=r"(w[i][j + 3]) : "l"(src + 4 * j));
        }
        asm volatile("ld.global.nc.u16 %0, [%1];" : "=h"(d[i]) : "l"(a.c.k_d + (row + r) * (D / 32) + (D == 128 ? t : t / 2)));
      }
    }
  }
};

// The steps' first pairs of a word as bf16 values, of 4 bits the numbers of bytes (0, 2), (1, 3) low, then high (two steps); of 8
// bits bytes (0, 1), (2, 3) (one step). As in kv_tile.cuh.
struct Scale4 {
  uint32_t dh, dl;
  __device__ __forceinline__ explicit Scale4(uint16_t d) {
    const float f = __half2float(__ushort_as_half(d));
    dh = pack_bf16x2(f, f);
    const float rest = f - __uint_as_float(dh << 16);
    dl = pack_bf16x2(rest, rest);
  }
  __device__ __forceinline__ uint32_t value(uint32_t nibbles) const {
    const uint32_t n = add_bf16x2((nibbles & 0x000f000fu) | 0x43004300u, 0xc308c308u);
    return fma_bf16x2(n, dh, mul_bf16x2(n, dl));
  }
  // ... and what is left of d n, which `value` rounds: n dh less that, and with n dl, have no more than seven bits each.
  __device__ __forceinline__ uint32_t value(uint32_t nibbles, uint32_t& rest) const {
    const uint32_t n = add_bf16x2((nibbles & 0x000f000fu) | 0x43004300u, 0xc308c308u), v = fma_bf16x2(n, dh, mul_bf16x2(n, dl));
    rest = fma_bf16x2(n, dl, fma_bf16x2(n, dh, v ^ 0x80008000u));
    return v;
  }
};
__device__ __forceinline__ uint32_t value_q8(uint32_t u, int k, uint64_t dd) {   // bytes k, k + 1, 128 more
  const uint64_t n = add_f32x2(f32x2(__uint_as_float(__byte_perm(u, 0x4B000000u, 0x7540u | k)),
                                     __uint_as_float(__byte_perm(u, 0x4B000000u, 0x7540u | (k + 1)))), f32x2(-8388736.f, -8388736.f));
  float lo, hi;
  f32x2_split(mul_f32x2(n, dd), lo, hi);
  return pack_bf16x2(lo, hi);
}
__device__ __forceinline__ uint32_t value_q8(uint32_t u, int k, uint64_t dd, uint32_t& rest) {   // ... and the rest of d n, rounded
  const uint64_t n = add_f32x2(f32x2(__uint_as_float(__byte_perm(u, 0x4B000000u, 0x7540u | k)),
                                     __uint_as_float(__byte_perm(u, 0x4B000000u, 0x7540u | (k + 1)))), f32x2(-8388736.f, -8388736.f));
  float lo, hi;
  f32x2_split(mul_f32x2(n, dd), lo, hi);
  const uint32_t v = pack_bf16x2(lo, hi);
  rest = pack_bf16x2(lo - __uint_as_float(v << 16), hi - __uint_as_float(v & 0xffff0000u));
  return v;
}

// NT * 8 rows at most, from row0 on. A warp has `runs` runs of 16 keys. STORED: keys are not rounded: of d n, a product of 11 and
// 4 (8) bits, the bf16 number and what that leaves, in 4 bits one as well, in 8 to 2^-17 of d n, are operands of two products, summed up
// apart (a token of 64 sequences of 1024 to 8192 keys, 32 heads on 8, D = 128: 110 us where rounded keys take 84, in 8 bits 131 and 91).
template <int D, bool Q4, bool PAGED, int NT, bool STORED>
__global__ void __launch_bounds__(128) weights_few_kernel(const __grid_constant__ WeightArgs a, int runs, unsigned chunks, unsigned warps, int row0) {
  constexpr int W = Quarter<D, Q4>::W, STEPS = D / 16;
  const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const unsigned id = blockIdx.x * 4 + (threadIdx.x >> 5);
  if (id >= warps) return;
  const unsigned bh = id / chunks;
  const int b = bh / a.c.Hkv, h = bh % a.c.Hkv, key0 = (int)(id % chunks) * runs * kRun;
  int len, n;
  read_lengths(a, b, id % chunks == 0 && h == 0 && lane == 0, len, n);
  const int before = len - n;   // the first token's position
  // the runs with a key that some token sees: [first, past)
  const int end = min(key0 + runs * kRun, len);
  const int first = max(key0, a.window > 0 ? max(before - a.window, 0) & ~(kRun - 1) : 0), past = n > 0 ? end : first;
  int entry = -1;   // lane i: the page of the chunk's run i
  if (PAGED && lane < runs && key0 + lane * kRun < past)
    entry = __ldg(a.pages.table + b * a.pages.stride + page_index(a.pages, key0 + lane * kRun));
  auto row_of = [&](int key) -> long long {
    if constexpr (!PAGED) return (long long)bh * a.c.S + key;
    return row_in_page(a.pages, __shfl_sync(0xffffffffu, entry, (key - key0) / kRun), a.c.Hkv, h, key, lane == 0 ? a.status : nullptr);
  };
  // Groups of four runs from the chunk's beginning; `from`: the first group with a run to do.
  const int from = key0 + ((first - key0) & ~(4 * kRun - 1));
  Quarter<D, Q4> ring[2];   // a run worked on, the next on its way
  auto load = [&](Quarter<D, Q4>& x, int key) {
    if (key < past) x.load(a, key < first ? -1 : row_of(key), past - key);
  };
  if (first < past) load(ring[0], from);

  // q: of row 8 m + g this lane's quarter, as the steps take it; of rows 8 m + 2 t and the next their LSE and position
  uint32_t q[NT][STEPS][2];
  float less[NT][2];
  int pos[NT][2];
#pragma unroll
  for (int m = 0; m < NT; ++m) {
    auto place = [&](int r) -> size_t {   // row of q, and of lse in one layout
      const int i = r / a.G, head = h * a.G + r % a.G;
      return a.layout ? ((size_t)b * a.Sq + i) * a.Hq + head : ((size_t)b * a.Hq + head) * a.Sq + i;
    };
    const int r = (STORED ? row0 : 0) + 8 * m + g;
    const bool on = first < past && r < n * a.G;
    const uint2* src = reinterpret_cast<const uint2*>(a.q + (on ? place(r) * D : 0));
#pragma unroll
    for (int j = 0; j < STEPS; ++j) {
      // the step's four features: of 4 bits those of the low, then of the high nibbles of word j / 2; of 8 bits of word j
      const int f = Q4 ? (D == 128 ? 32 * t + 4 * (j / 2) : 32 * (t / 2) + 8 * (t & 1) + 4 * (j / 2)) + 16 * (j & 1) : (D / 4) * t + 4 * j;
      const uint2 x = on ? __ldg(src + f / 4) : make_uint2(0, 0);
      q[m][j][0] = Q4 ? __byte_perm(x.x, x.y, 0x5410) : x.x;
      q[m][j][1] = Q4 ? __byte_perm(x.x, x.y, 0x7632) : x.y;
    }
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int c = (STORED ? row0 : 0) + 8 * m + 2 * t + j;
      const bool live = c < n * a.G;
      const int i = c / a.G, head = h * a.G + c % a.G;
      less[m][j] = live && first < past ? -__ldg(a.lse + ((size_t)b * a.Hq + head) * a.Sq + i) * kLog2e : -CUDART_INF_F;
      pos[m][j] = live ? before + i : -1;
    }
  }

  float* out = a.out + (size_t)bh * a.W;
  const float* weights = a.weights != nullptr ? a.weights + (size_t)bh * a.W : nullptr;
  auto step = [&](const Quarter<D, Q4>& x, int key, float& kept0, float& kept1, bool keep) {
    float c[NT][4];
#pragma unroll
    for (int m = 0; m < NT; ++m) c[m][0] = c[m][1] = c[m][2] = c[m][3] = 0.f;
    if constexpr (STORED) {
      float rest[NT][4];
#pragma unroll
      for (int m = 0; m < NT; ++m) rest[m][0] = rest[m][1] = rest[m][2] = rest[m][3] = 0.f;
      // a step: the pairs of both rows, and their products with the step's pairs of q
      auto product = [&](int j, const uint32_t (&v)[4], const uint32_t (&w)[4]) {
#pragma unroll
        for (int m = 0; m < NT; ++m) {
          mma_bf16(c[m], v[0], v[1], v[2], v[3], q[m][j][0], q[m][j][1]);
          mma_bf16(rest[m], w[0], w[1], w[2], w[3], q[m][j][0], q[m][j][1]);
        }
      };
      uint32_t v[4], w[4];
      if constexpr (Q4) {
        const Scale4 d0(x.d[0]), d1(x.d[1]);
#pragma unroll
        for (int j = 0; j < W; ++j) {
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            const uint32_t r0 = x.w[0][j] >> (4 * half), r1 = x.w[1][j] >> (4 * half);
            v[0] = d0.value(r0, w[0]);
            v[1] = d1.value(r1, w[1]);
            v[2] = d0.value(r0 >> 8, w[2]);
            v[3] = d1.value(r1 >> 8, w[3]);
            product(2 * j + half, v, w);
          }
        }
      } else {
        const float f0 = __half2float(__ushort_as_half(x.d[0])), f1 = __half2float(__ushort_as_half(x.d[1]));
        const uint64_t d0 = f32x2(f0, f0), d1 = f32x2(f1, f1);
#pragma unroll
        for (int j = 0; j < W; ++j) {
          const uint32_t r0 = x.w[0][j] ^ 0x80808080u, r1 = x.w[1][j] ^ 0x80808080u;
          v[0] = value_q8(r0, 0, d0, w[0]);
          v[1] = value_q8(r1, 0, d1, w[1]);
          v[2] = value_q8(r0, 2, d0, w[2]);
          v[3] = value_q8(r1, 2, d1, w[3]);
          product(j, v, w);
        }
      }
#pragma unroll
      for (int m = 0; m < NT; ++m)
#pragma unroll
        for (int j = 0; j < 4; ++j) c[m][j] += rest[m][j];
    } else if constexpr (Q4) {
      const Scale4 d0(x.d[0]), d1(x.d[1]);
#pragma unroll
      for (int j = 0; j < W; ++j) {
        const uint32_t u = x.w[0][j], v = x.w[1][j];
        const uint32_t u0 = d0.value(u), u1 = d0.value(u >> 8), v0 = d1.value(v), v1 = d1.value(v >> 8);
        const uint32_t u2 = d0.value(u >> 4), u3 = d0.value(u >> 12), v2 = d1.value(v >> 4), v3 = d1.value(v >> 12);
#pragma unroll
        for (int m = 0; m < NT; ++m) {
          mma_bf16(c[m], u0, v0, u1, v1, q[m][2 * j][0], q[m][2 * j][1]);
          mma_bf16(c[m], u2, v2, u3, v3, q[m][2 * j + 1][0], q[m][2 * j + 1][1]);
        }
      }
    } else {
      const float f0 = __half2float(__ushort_as_half(x.d[0])), f1 = __half2float(__ushort_as_half(x.d[1]));
      const uint64_t d0 = f32x2(f0, f0), d1 = f32x2(f1, f1);
#pragma unroll
      for (int j = 0; j < W; ++j) {
        const uint32_t u = x.w[0][j] ^ 0x80808080u, v = x.w[1][j] ^ 0x80808080u;
        const uint32_t u0 = value_q8(u, 0, d0), u1 = value_q8(u, 2, d0), v0 = value_q8(v, 0, d1), v1 = value_q8(v, 2, d1);
#pragma unroll
        for (int m = 0; m < NT; ++m) mma_bf16(c[m], u0, v0, u1, v1, q[m][j][0], q[m][j][1]);
      }
    }
    const bool edge = key + kRun - 1 > before || (a.window > 0 && before + n - 1 - key > a.window);   // some token does not see all 16
    float sum[2] = {0.f, 0.f};
#pragma unroll
    for (int m = 0; m < NT; ++m)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        float p = ex2_approx(fmaf(c[m][j], a.sl2, less[m][j & 1]));
        if (edge) {
          const int k = key + g + 8 * (j >> 1), at = pos[m][j & 1];
          if (k > at || (a.window > 0 && at - k > a.window)) p = 0.f;
        }
        sum[j >> 1] += p;
      }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      sum[i] += __shfl_xor_sync(0xffffffffu, sum[i], 1);
      sum[i] += __shfl_xor_sync(0xffffffffu, sum[i], 2);
    }
    if (keep) {
      kept0 = sum[0];
      kept1 = sum[1];
    }
  };
  // Lane (g, t) has what there was, and what is added, of keys g and g + 8 of run t of a group.
  const int all = (int)min((long long)key0 + runs * kRun, a.W);
  for (int key = key0; key < all; key += 4 * kRun) {
    const int k0 = key + kRun * t + g, k1 = k0 + 8;
    const float had0 = weights != nullptr && k0 < all ? weights[k0] : 0.f, had1 = weights != nullptr && k1 < all ? weights[k1] : 0.f;
    float sum0 = 0.f, sum1 = 0.f;
    if (key >= from && key < past) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int at = key + i * kRun;
        if (at >= past) break;
        load(ring[(i + 1) & 1], at + kRun);
        if (at >= first) step(ring[i & 1], at, sum0, sum1, t == i);
      }
    }
    if (k0 < all) out[k0] = had0 + sum0;
    if (k1 < all) out[k1] = had1 + sum1;
  }
}

constexpr int kUnit = 2 * kTileKeys;   // keys of a block at a time
constexpr int kRows = 128;             // rows of a tile
constexpr int kUnits = 4;              // descriptions of units in shared memory

// What the roles of a block know of 256 keys and the rows that see one of them: rows [row0, row0 + rows) of the key/value head.
struct Unit { int b, h, key0, before, row0, rows, padding[2]; };

template <int D>
struct WeightSmem {
  static constexpr int kBox = 128 * 128;            // 64 features of 128 rows
  static constexpr int kTile = 128 * D * 2;
  static constexpr int kRing = 3;                   // tiles of rows
  static constexpr int kQOff = 4 * kTile;           // two units of keys
  static constexpr int kLogOff = kQOff + kRing * kTile, kSumOff = kLogOff + kRing * kRows * 4, kBarOff = kSumOff + kUnit * 4;
  static constexpr int kBytes = kBarOff + 512;
};

template <int D, bool Q4, bool PAGED>
__global__ void __launch_bounds__(kThreads, 1) weights_kernel(const __grid_constant__ WeightArgs a, unsigned total) {
  using L = WeightSmem<D>;
  extern __shared__ __align__(1024) uint8_t smem[];
  const uint32_t sK = smem_u32(smem), sQ = smem_u32(smem + L::kQOff);
  float* sLog = reinterpret_cast<float*>(smem + L::kLogOff);   // [ring][128]: -lse, base 2; -inf in columns without a row
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + L::kBarOff);
  uint64_t* bar_k = bars;               // [2]: a unit's K written
  uint64_t* bar_kfree = bars + 2;       // [2]: its products done
  uint64_t* bar_q = bars + 4;           // [ring]: rows written
  uint64_t* bar_qfree = bars + 7;       // [ring]: products done
  uint64_t* bar_log = bars + 10;        // [ring]: the rows' LSE read
  uint64_t* bar_s = bars + 13;          // [2 tiles of keys][2]: products there
  uint64_t* bar_sfree = bars + 17;      // [2][2]: read
  uint64_t* bar_unit = bars + 21;       // [kUnits]: described
  uint64_t* bar_done = bars + 25;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 26);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  Unit* units = reinterpret_cast<Unit*>(smem + L::kBarOff + 256);
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const unsigned heads = (unsigned)a.c.B * a.c.Hkv;

  if (threadIdx.x == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bar_k[i], kLoaders);
      mbar_init(&bar_kfree[i], 1);
    }
    for (int i = 0; i < L::kRing; ++i) {
      mbar_init(&bar_q[i], kLoaders);
      mbar_init(&bar_qfree[i], 1);
      mbar_init(&bar_log[i], 16);   // the warps that add
    }
    for (int i = 0; i < 4; ++i) {
      mbar_init(&bar_s[i], 1);
      mbar_init(&bar_sfree[i], 8);
      mbar_init(&bar_unit[i], 1);
    }
    mbar_init(bar_done, 1);
    *abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == 0) tmem_alloc(tmem_slot, 512);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, *tmem_slot, 0);
  // Unit i of those with rows is described; one without rows is the end. A description is read when its unit begins: it is
  // written over for unit i + 4, when unit i + 2 is done, whose last products came after unit i's had been taken.
  auto unit_there = [&](int i) { return mbar_wait_warp(&bar_unit[i % kUnits], (i / kUnits) & 1, abort_flag, a.status, 1101); };

  if (warp < 8) regs_inc<kRegsLoad>();
  else regs_dec<kRegsAdd>();
  if (warp == 0) {
    // ------------------------------------------------------------------ MMAs, the lanes together
    const uint32_t lead = lane == 0 ? 1u : 0u, idesc = idesc_bf16_f32(128, kRows, 0, 0);
    const uint64_t dk = smem_desc_sw128(sK, 16, 1024), dq = smem_desc_sw128(sQ, 16, 1024);
    bool ok = true;
    int x = 0, slot = 0, laps = 0;   // tiles of rows so far; of the ring: the place, and how often it has gone round
    for (int i = 0; ok; ++i) {
      if (!(ok = unit_there(i))) break;
      const int rows = __shfl_sync(0xffffffffu, units[i % kUnits].rows, 0);
      if (rows == 0) break;
      if (!(ok = mbar_wait_warp(&bar_k[i & 1], (i >> 1) & 1, abort_flag, a.status, 1102))) break;
      for (int r = 0; ok && r < rows; r += kRows, ++x) {
        if (!(ok = mbar_wait_warp(&bar_q[slot], laps & 1, abort_flag, a.status, 1103))) break;
        for (int m = 0; ok && m < 2; ++m) {
          const int buf = 2 * m + (x & 1);
          if (x >= 2 && !(ok = mbar_wait_warp(&bar_sfree[buf], ((x >> 1) - 1) & 1, abort_flag, a.status, 1104))) break;
          tc_fence_after();
          const uint64_t k0 = desc_add(dk, (2 * (i & 1) + m) * L::kTile), q0 = desc_add(dq, slot * L::kTile);
#pragma unroll
          for (int k = 0; k < D / 16; ++k)
            mma_ss_if(lead, tmem + buf * kRows, desc_add(k0, (k >> 2) * L::kBox + (k & 3) * 32), desc_add(q0, (k >> 2) * L::kBox + (k & 3) * 32),
                      idesc, k > 0 ? 1u : 0u);
          mma_commit_if(lead, &bar_s[buf]);
        }
        if (!ok) break;
        mma_commit_if(lead, &bar_qfree[slot]);
        if (++slot == L::kRing) {
          slot = 0;
          ++laps;
        }
      }
      if (ok) mma_commit_if(lead, &bar_kfree[i & 1]);
    }
    mma_commit_if(lead, bar_done);
    mbar_wait<true>(bar_done, 0, nullptr, a.status, 1105);
    __syncwarp();
  } else if (warp < 8) {
    // ------------------------------------------------------------------ the units, their K, and the rows: a part of each for every warp
    constexpr int CHUNKS = D / 8, ROWS = 32 / CHUNKS, STEP = kLoaders * ROWS;   // 16-byte chunks of a row, rows of a load, of a step
    const int w = warp - 1, me = w * 32 + lane;
    const int chunk = lane % CHUNKS, r0 = w * ROWS + lane / CHUNKS;
    const int tokens = STEP / a.G, over_heads = STEP % a.G;
    const long long by_token = (long long)(a.layout ? a.Hq : 1) * D, by_head = (long long)(a.layout ? 1 : a.Sq) * D;
    const long long on_by = tokens * by_token + over_heads * by_head, over = by_token - a.G * by_head;
    int slot = 0, laps = 0;
    int last = -1, last_rows = 0;   // the tile before, of which the copies are still on their way: its place, and its rows
    bool ok = true;
    unsigned id = blockIdx.x;
    int units_so_far = 0, len = 0;
    // The next unit with rows, its place described, its K made; the end where there is none. It takes the place of the unit two
    // before, whose products have to be done.
    auto next_unit = [&](Unit& u) -> bool {
      u.rows = 0;
      for (; id < total && u.rows == 0; id += gridDim.x) {
        const int bh = id % heads, b = bh / a.c.Hkv, h = bh % a.c.Hkv, key0 = (int)(id / heads) * kUnit;
        int n;
        read_lengths(a, b, key0 == 0 && h == 0 && me == 0, len, n);
        const int before = len - n, first = max(key0 - before, 0);   // tokens [first, past) see one of the keys
        const int past = a.window > 0 ? min(n, min(key0 + kUnit, len) + a.window - before) : n;
        u = Unit{b, h, key0, before, first * a.G, key0 < len ? max(past - first, 0) * a.G : 0, {0, 0}};
        if (u.rows == 0) {   // nobody sees them
          for (int k = me; k < kUnit; k += 32 * kLoaders) {
            const size_t at = (size_t)bh * a.W + key0 + k;
            if (key0 + k < a.W) a.out[at] = a.weights != nullptr ? a.weights[at] : 0.f;
          }
        }
      }
      const int i = units_so_far++;
      if (i >= 2 && !(ok = mbar_wait_warp(&bar_kfree[i & 1], ((i >> 1) - 1) & 1, abort_flag, a.status, 1107))) return false;
      if (me == 0) {
        units[i % kUnits] = u;
        mbar_arrive(&bar_unit[i % kUnits]);
      }
      if (u.rows == 0) return false;
      RunBytes<D, Q4> k[2];
      auto load = [&](RunBytes<D, Q4>& x, int r) {
        if (r >= kUnit / kRun) return;
        const int run = u.key0 + kRun * r;
        long long row = -1;
        if (run < len) row = PAGED ? page_row(a.pages, a.c.Hkv, u.b, u.h, run, lane == 0 ? a.status : nullptr) : ((long long)u.b * a.c.Hkv + u.h) * a.c.S + run;
        x.load(a.c.k_q, a.c.k_d, row, len - run);
      };
      auto store = [&](const RunBytes<D, Q4>& x, int r) {
        if (r < kUnit / kRun) x.store(sK + (2 * (i & 1) + r / 8) * L::kTile, r % 8, false);
      };
      static_assert(kUnit / kRun <= 3 * kLoaders, "a warp has three runs at most");
      load(k[0], w);
      load(k[1], w + kLoaders);
      store(k[0], w);
      load(k[0], w + 2 * kLoaders);
      store(k[1], w + kLoaders);
      store(k[0], w + 2 * kLoaders);
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bar_k[i & 1]);
      return true;
    };
    auto complete = [&] {
      for (int r = me; r < kRows; r += 32 * kLoaders) {
        float& x = sLog[last * kRows + r];
        x = r < last_rows ? -x * kLog2e : -CUDART_INF_F;
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bar_q[last]);
      last = -1;
    };
    Unit u, then;
    bool has = next_unit(u);
    while (has && ok) {
      bool prepared = false, more = false;
      for (int first = 0; first < u.rows; first += kRows) {
        if (laps > 0) {
          if (last >= 0 && !__all_sync(0xffffffffu, mbar_test(&bar_qfree[slot], (laps - 1) & 1) && mbar_test(&bar_log[slot], (laps - 1) & 1))) {
            asm volatile("cp.async.wait_all;" ::: "memory");   // no place yet: see the last tile in first
            complete();
          }
          if (!(ok = mbar_wait_warp(&bar_qfree[slot], (laps - 1) & 1, abort_flag, a.status, 1106))) break;
          if (!(ok = mbar_wait_warp(&bar_log[slot], (laps - 1) & 1, abort_flag, a.status, 1109))) break;
        }
        const int rows = u.rows - first, row = u.row0 + first + r0;
        int head = row % a.G;
        const __nv_bfloat16* src = a.q + ((size_t)u.b * a.Hq * a.Sq) * D + (row / a.G) * by_token + (u.h * a.G + head) * by_head + 8 * chunk;
        const uint32_t box = sQ + slot * L::kTile + (chunk >> 3) * L::kBox;
#pragma unroll 2
        for (int r = r0; r < kRows; r += STEP) {   // rows behind the last are zeros
          const bool on = r < rows;
          asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(box + r * 128 + (((chunk & 7) ^ (r & 7)) << 4)),
                       "l"(on ? src : a.q), "r"(on ? 16 : 0) : "memory");
          src += on_by;
          head += over_heads;
          if (head >= a.G) {
            head -= a.G;
            src += over;
          }
        }
        for (int r = me; r < min(rows, kRows); r += 32 * kLoaders) {
          const int at = u.row0 + first + r;
          asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem_u32(sLog + slot * kRows + r)),
                       "l"(a.lse + ((size_t)u.b * a.Hq + u.h * a.G + at % a.G) * a.Sq + at / a.G) : "memory");
        }
        asm volatile("cp.async.commit_group;\n\tcp.async.wait_group 1;" ::: "memory");
        if (last >= 0) complete();
        last = slot;
        last_rows = rows;
        if (++slot == L::kRing) {
          slot = 0;
          ++laps;
        }
        // The next unit when this one's fourth tile is on its way: the products of the one before are done then, as the first
        // tile's place was free. Where there are not so many tiles, they are all there before it is waited for that.
        if (!prepared && (first == 3 * kRows || first + kRows >= u.rows)) {
          if (first < 3 * kRows) {
            asm volatile("cp.async.wait_all;" ::: "memory");
            complete();   // the last tile, just asked for
          }
          more = next_unit(then);
          prepared = true;
        }
      }
      u = then;
      has = more;
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
    if (last >= 0) complete();
  } else {
    // ------------------------------------------------------------------ exponentials and sums: a key, and half of the rows, for each thread
    const int m = (warp - 8) / 8, half = (warp - 8) / 4 & 1, wq = warp & 3;
    const uint32_t tS = tmem + 2 * m * kRows + half * 64 + ((uint32_t)(wq * 32) << 16);
    const uint64_t sl2 = f32x2(a.sl2, a.sl2);
    float* sums = reinterpret_cast<float*>(smem + L::kSumOff) + m * kTileKeys + wq * 32 + lane;   // what the second half's thread has
    const int pair = 1 + m * 4 + wq;   // the barrier of the two warps that have the same keys: they go the same way, in what fails too
    int x = 0, slot = 0;
    for (int i = 0;; ++i) {
      bool ok = named_bar_and(pair, 64, unit_there(i));
      const Unit u = units[i % kUnits];
      if (!ok || u.rows == 0) break;
      const int key = u.key0 + m * kTileKeys + wq * 32 + lane;
      const size_t at = ((size_t)u.b * a.c.Hkv + u.h) * a.W + key;
      const float had = half == 0 && a.weights != nullptr && key < a.W ? a.weights[at] : 0.f;
      float sum = 0.f;
      for (int first = 0; first < u.rows; first += kRows, ++x) {
        const int buf = x & 1, here = min(u.rows - first - half * 64, 64);   // columns with a row
        if (!(ok = mbar_wait_warp(&bar_s[2 * m + buf], (x >> 1) & 1, abort_flag, a.status, 1108))) break;
        tc_fence_after();
        const float* log = sLog + slot * kRows + half * 64;
        const int row = u.row0 + first + half * 64;
        int pos = u.before + row / a.G, head = row % a.G;   // of the column at hand
        const int pos1 = u.before + (row + here - 1) / a.G;   // of the last one
        const bool edge = pos < u.key0 + (m + 1) * kTileKeys - 1 || (a.window > 0 && pos1 - (u.key0 + m * kTileKeys) > a.window);
        uint64_t part[2] = {f32x2(0.f, 0.f), f32x2(0.f, 0.f)};
        auto add = [&](int c0, auto on_edge) {
          uint32_t raw[32];
          tmem_ld32(tS + buf * kRows + c0, raw);
          tmem_wait_ld();
          reg_fence(raw);
#pragma unroll
          for (int e = 0; e < 32; e += 4) {
            const float4 g = *reinterpret_cast<const float4*>(log + c0 + e);
            float p[4];
            f32x2_split(fma_f32x2(f32x2(__uint_as_float(raw[e]), __uint_as_float(raw[e + 1])), sl2, f32x2(g.x, g.y)), p[0], p[1]);
            f32x2_split(fma_f32x2(f32x2(__uint_as_float(raw[e + 2]), __uint_as_float(raw[e + 3])), sl2, f32x2(g.z, g.w)), p[2], p[3]);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              p[k] = ex2_approx(p[k]);
              if constexpr (decltype(on_edge)::value) {   // hidden: no weight, whatever came out
                if (key > pos || (a.window > 0 && pos - key > a.window)) p[k] = 0.f;
                if (++head == a.G) {
                  head = 0;
                  ++pos;
                }
              }
            }
            part[0] = add_f32x2(part[0], f32x2(p[0], p[1]));
            part[1] = add_f32x2(part[1], f32x2(p[2], p[3]));
          }
        };
        if (edge) {
#pragma unroll 1
          for (int c0 = 0; c0 < here; c0 += 32) add(c0, std::true_type{});
        } else {
#pragma unroll 1
          for (int c0 = 0; c0 < here; c0 += 32) add(c0, std::false_type{});
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(&bar_sfree[2 * m + buf]);
          mbar_arrive(&bar_log[slot]);
        }
        slot = slot == L::kRing - 1 ? 0 : slot + 1;
        float s0, s1, s2, s3;
        f32x2_split(part[0], s0, s1);
        f32x2_split(part[1], s2, s3);
        sum += (s0 + s1) + (s2 + s3);
      }
      if (half == 1) *sums = sum;
      if (!named_bar_and(pair, 64, ok)) break;
      if (half == 0 && key < a.W) a.out[at] = had + (sum + *sums);
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 0) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

template <int D, bool Q4, bool PAGED, int NT, bool STORED>
fa_status launch_weights_few(const WeightArgs& a, long long heads, cudaStream_t st, int row0 = 0) {
  // 256 keys a warp, so that what comes before the first costs little, where that leaves eight warps for each SM at least, else 64
  // (groups of four runs). In 4 bits, D = 128, 8 heads, with 256 and with 64, of 4 rows and of 16: 64 sequences of 1024 to 8192 keys
  // 83.5 and 93.6 us, 107 and 130; one of 67,584 22.1 and 21.2, 25.9 and 29.7; 16 of 1024 to 4096 21.4 and 16.4, 25.2 and 22.0 (fourteen
  // warps an SM, of different lengths); 8 of 1000 to 4000 (seven) 17.5 and 10.0, 17.8 and 13.8; 2 of 500 to 1000 12.1 and 5.5, 13.7 and 6.9.
  const int runs = heads * ((a.W + 255) / 256) >= 8LL * sm_count() ? 16 : 4;
  const long long chunks = (a.W + runs * kRun - 1) / (runs * kRun), warps = heads * chunks;
  if (warps > 0x7fffffffLL) return cuda_status(cudaErrorInvalidConfiguration, "cache weights launch");
  weights_few_kernel<D, Q4, PAGED, NT, STORED><<<(unsigned)((warps + 3) / 4), 128, 0, st>>>(a, runs, (unsigned)chunks, (unsigned)warps, row0);
  count_launches(1);
  return cuda_status(cudaGetLastError(), "cache weights launch");
}

template <int D, bool Q4, bool PAGED>
fa_status launch_weights(const WeightArgs& a, long long heads, cudaStream_t st) {
  constexpr int bytes = WeightSmem<D>::kBytes;
  static_assert(bytes <= 232448, "shared memory of a block");
  auto kernel = weights_kernel<D, Q4, PAGED>;
  static std::atomic<uint64_t> allowed{0};
  if (allowed.load(std::memory_order_acquire) == 0) {
    const fa_status got = check_split(kernel, "cache weights launch", kRegsLaunch);
    if (got != FA_OK) return got;
  }
  const cudaError_t e = allow_shared(kernel, bytes, allowed);
  if (e != cudaSuccess) return cuda_status(e, "cache weights launch");
  const long long total = heads * ((a.W + kUnit - 1) / kUnit);
  if (total > 0x7fffffffLL) return cuda_status(cudaErrorInvalidConfiguration, "cache weights launch");
  const unsigned blocks = (unsigned)(total < sm_count() ? total : sm_count());
  kernel<<<blocks, kThreads, bytes, st>>>(a, (unsigned)total);
  count_launches(1);
  return cuda_status(cudaGetLastError(), "cache weights launch");
}

}  // namespace
}  // namespace fa

using namespace fa;

namespace {

// stored: the LSE was made with keys as they are stored, which then are not rounded.
fa_status key_weights(const fa_prefill_params* p, const void* q, const float* lse, const fa_cache* c, const fa_pages* pages,
                      const int64_t* lengths, const int64_t* count, const float* weights, int64_t W, float* out, bool stored,
                      void* stream) {
  CacheView held, cv;
  PageView pv;
  Span in[8], planes[4], outs[1];
  fa_status st = check_paged(c, pages, held, cv, pv, in[4]);
  if (st != FA_OK) return st;
  if ((st = check_chunk(p, cv)) != FA_OK) return st;
  const long long heads = (long long)cv.B * cv.Hkv;
  if (W < 1 || W > 1LL << 30) { set_error("W=%lld outside [1, 2^30]", (long long)W); return FA_ERR_INVALID_ARG; }
  if ((W + 63) / 64 * heads > 0x7fffffffLL) { set_error("too many keys for one launch"); return FA_ERR_UNSUPPORTED; }   // of 64 at least
  const size_t rows = (size_t)cv.B * p->Hq * p->Sq, bytes = (size_t)heads * (size_t)W * 4;
  cache_spans(held, planes);
  in[0] = planes[0];
  in[1] = planes[1];
  in[2] = {q, rows * cv.D * 2, "q"};
  in[3] = {lse, rows * 4, "lse"};
  outs[0] = {out, bytes, "out"};
  const Span table = in[4];
  if ((st = check_buffers(in, 4, outs, 1)) != FA_OK) return st;
  in[4] = table;
  in[5] = {lengths, lengths != nullptr ? (size_t)cv.B * 8 : 0, "lengths"};
  in[6] = {count, count != nullptr ? (size_t)cv.B * 8 : 0, "count"};
  in[7] = {weights, weights != nullptr && weights != out ? bytes : 0, "weights"};
  if ((uintptr_t)lengths % 8 != 0 || (uintptr_t)count % 8 != 0) {
    set_error("lengths and count must be 8-byte aligned"); return FA_ERR_INVALID_ARG;
  }
  if ((uintptr_t)weights % 16 != 0) { set_error("weights is not 16-byte aligned"); return FA_ERR_INVALID_ARG; }
  if ((st = check_apart(in + 4, 4, outs, 1)) != FA_OK) return st;
  WeightArgs a{};
  a.c = cv;
  a.pages = pv;
  a.q = static_cast<const __nv_bfloat16*>(q);
  a.lse = lse;
  a.lengths = lengths;
  a.count = count;
  a.weights = weights;
  a.out = out;
  if ((a.status = device_status_ptr()) == nullptr) return cuda_status(cudaErrorUnknown, "status word");
  a.W = W;
  a.sl2 = fmaxf(fminf(p->scale * kLog2e, FLT_MAX), -FLT_MAX);
  a.Hq = p->Hq;
  a.Sq = p->Sq;
  a.window = p->window < 2 * kMaxSeq ? p->window : 2 * kMaxSeq;
  a.layout = p->layout;
  a.G = p->Hq / cv.Hkv;
  const long long rows_of_head = (long long)a.G * p->Sq;
  auto go = [&](auto dim, auto q4) {
    constexpr int D = decltype(dim)::value;
    constexpr bool Q4 = decltype(q4)::value;
    cudaStream_t cs = (cudaStream_t)stream;
    auto of = [&](auto paged) {
      constexpr bool P = decltype(paged)::value;
      if (stored) {   // 16 rows after the other, each launch's weights on top of the last one's
        WeightArgs x = a;
        for (long long row0 = 0;; row0 += 16) {
          const bool few = rows_of_head - row0 <= 8;
          const fa_status got = few ? launch_weights_few<D, Q4, P, 1, true>(x, heads, cs, (int)row0)
                                    : launch_weights_few<D, Q4, P, 2, true>(x, heads, cs, (int)row0);
          if (got != FA_OK || row0 + 16 >= rows_of_head) return got;
          x.weights = x.out;
        }
      }
      // Up to 16 rows by way of registers, more by tcgen05 tiles: a step of 64 sequences of 1024 to 8192 keys, 8 heads, D = 128, takes
      // with 4, 8 and 16 rows 83, 84 and 107 us against 295 to 297 in 4 bits, 91, 92 and 109 against 347 to 352 in 8; one sequence of
      // 67,584 keys 22 (4 rows) and 26 (16) against 60. The two meet further on: 20, 24 and 32 rows (which are not built) 148, 148 and
      // 168 against 300, and 42 to 47 against 60.
      if (rows_of_head <= 8) return launch_weights_few<D, Q4, P, 1, false>(a, heads, cs);
      if (rows_of_head <= 16) return launch_weights_few<D, Q4, P, 2, false>(a, heads, cs);
      return launch_weights<D, Q4, P>(a, heads, cs);
    };
    return pages != nullptr ? of(std::true_type{}) : of(std::false_type{});
  };
  using D64 = std::integral_constant<int, 64>;
  using D128 = std::integral_constant<int, 128>;
  if (cv.q4) return cv.D == 64 ? go(D64{}, std::true_type{}) : go(D128{}, std::true_type{});
  return cv.D == 64 ? go(D64{}, std::false_type{}) : go(D128{}, std::false_type{});
}

}  // namespace

extern "C" {

fa_status fa_cache_weights(const fa_prefill_params* p, const void* q, const float* lse, const fa_cache* c, const fa_pages* pages,
                           const int64_t* lengths, const int64_t* count, const float* weights, int64_t W, float* out,
                           void* stream) {
  clear_error();
  if (p == nullptr) { set_error("params is NULL"); return FA_ERR_INVALID_ARG; }
  return key_weights(p, q, lse, c, pages, lengths, count, weights, W, out, false, stream);
}

fa_status fa_cache_weights_decoded(const fa_decode_params* p, const void* q, const float* lse, const fa_cache* c,
                                   const fa_pages* pages, const int64_t* lengths, const float* weights, int64_t W, float* out,
                                   void* stream) {
  clear_error();
  if (p == nullptr) { set_error("params is NULL"); return FA_ERR_INVALID_ARG; }
  if (p->Sq > kDecodeTokens) { set_error("Sq=%d outside [0, %d]", p->Sq, kDecodeTokens); return FA_ERR_INVALID_ARG; }
  const fa_prefill_params x{p->Hq, p->Sq, p->window, p->layout, p->scale, p->reserved};
  return key_weights(&x, q, lse, c, pages, lengths, nullptr, weights, W, out, true, stream);
}

}  // extern "C"
