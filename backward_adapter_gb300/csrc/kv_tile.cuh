// A tile of 128 keys of a quantized plane as the bf16 operand of tcgen05.mma: eight warps read a run of 16 rows each, 16 bytes a
// lane and load, and write them in the 128-byte-swizzled layout that TMA would have written (64-feature boxes of 128 rows x 128
// bytes, 16-byte chunk c of row r at chunk c ^ (r & 7)). Eight neighbouring lanes hold eight rows, so that their stores meet
// no bank twice.
//
// A value is bf16(d n), rounded once. 8 bits: d n is exact in fp32. 4 bits, two values an instruction: d = dh + dl with dh =
// bf16(d), whose error dl has two bits at most (d has 11, dh 8 of them); n dl then is exact in bf16, and n dh + n dl in one
// fused operation is d n rounded once. n itself comes as the mantissa of 128 + (n + 8), an exact subtraction away.
#pragma once

#include <cuda_fp16.h>
#include <stdint.h>

#include "kv_pages.cuh"
#include "kv_q8.cuh"
#include "tc_ptx.cuh"

namespace fa {

constexpr int kTileKeys = 128;
constexpr int kRun = 16;   // keys of a run: they lie in one page

__device__ __forceinline__ uint32_t add_bf16x2(uint32_t x, uint32_t y) {
  uint32_t z;
  asm("add.rn.bf16x2 %0, %1, %2;" : "=r"(z) : "r"(x), "r"(y));
  return z;
}
__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t x, uint32_t y) {
  uint32_t z;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(z) : "r"(x), "r"(y));
  return z;
}
__device__ __forceinline__ uint32_t fma_bf16x2(uint32_t x, uint32_t y, uint32_t a) {
  uint32_t z;
  asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(z) : "r"(x), "r"(y), "r"(a));
  return z;
}

// The bytes of a run, in a warp's registers.
template <int D, bool Q4>
struct RunBytes {
  static constexpr int ROW = Q4 ? D / 2 : D;    // bytes of a row
  static constexpr int PIECES = ROW / 16;
  static constexpr int N = kRun * PIECES / 32;  // loads of a lane
  static constexpr int NB = D / 32;
  static constexpr int BOX = 128 * 128;         // bytes of a 64-feature box of the tile
  uint32_t w[N][4];
  uint16_t d[N];

  // Load i: the lane's row of the run, and which piece of it.
  __device__ static __forceinline__ int row_of(int i, int lane) {
    return PIECES == 2 ? 8 * (lane >> 4) + (lane & 7) : PIECES == 4 ? 8 * i + (lane & 7) : 8 * (i >> 1) + (lane & 7);
  }
  __device__ static __forceinline__ int piece_of(int i, int lane) {
    return PIECES == 2 ? (lane >> 3) & 1 : PIECES == 4 ? lane >> 3 : 4 * (i & 1) + (lane >> 3);
  }

  // The first `keys` rows from row `first` of a plane on; the others, and all where that is negative, are zeros, and not
  // read. The loads stay in this place among the waits.
  __device__ __forceinline__ void load(const void* values, const uint16_t* scales, long long first, int keys) {
    const int lane = threadIdx.x & 31;
    const int at = row_of(0, lane) * ROW + 16 * piece_of(0, lane), scale_at = row_of(0, lane) * NB + piece_of(0, lane) / (Q4 ? 1 : 2);
    const uint8_t* v = static_cast<const uint8_t*>(values) + first * ROW + at;
    const uint16_t* s = scales + first * NB + scale_at;
    if (first < 0) keys = 0;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int rows = PIECES == 4 ? 8 * i : PIECES == 8 ? 8 * (i >> 1) : 0, more = PIECES == 8 ? 4 * (i & 1) : 0;   // of the first load
      w[i][0] = w[i][1] = w[i][2] = w[i][3] = Q4 ? 0x88888888u : 0u;
      d[i] = 0;
      if (row_of(i, lane) < keys) {
        asm volatile("ld.global.nc.L1::no_allocate.v4.b32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(w[i][0]), "=r"(w[i][1]), "=r"(w[i][2]), "=r"(w[i][3]) : "l"(v + rows * ROW + 16 * more));
        asm volatile("ld.global.nc.L1::no_allocate.u16 %0, [%1];" : "=h"(d[i]) : "l"(s + rows * NB + more / 2));
      }
    }
  }

  // Into run `run` of the tile at `tile` (shared memory). finite: a scale that is not counts as 0.
  __device__ __forceinline__ void store(uint32_t tile, int run, bool finite) const {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int piece = piece_of(i, lane);
      float df = __half2float(__ushort_as_half(d[i]));
      if (finite && !(fabsf(df) <= 65504.f)) df = 0.f;
      const uint32_t at = tile + (kRun * run + row_of(i, lane)) * 128;
      auto put = [&](int chunk, uint32_t a, uint32_t b, uint32_t c, uint32_t e) {
        tc::st_shared_v4(at + (chunk >> 3) * BOX + (((chunk & 7) ^ (lane & 7)) << 4), a, b, c, e);
      };
      if constexpr (Q4) {
        const uint32_t dh = tc::pack_bf16x2(df, df);
        const float rest = df - __uint_as_float(dh << 16);
        const uint32_t dl = tc::pack_bf16x2(rest, rest);
        auto value = [&](uint32_t bytes) {   // of the low nibbles of two bytes, 16 bits apart
          const uint32_t n = add_bf16x2((bytes & 0x000f000fu) | 0x43004300u, 0xc308c308u);
          return fma_bf16x2(n, dh, mul_bf16x2(n, dl));
        };
        uint32_t lo[8], hi[8];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const uint32_t x = __byte_perm(w[i][j], 0u, 0x4140), y = __byte_perm(w[i][j], 0u, 0x4342);
          lo[2 * j] = value(x);
          lo[2 * j + 1] = value(y);
          hi[2 * j] = value(x >> 4);
          hi[2 * j + 1] = value(y >> 4);
        }
        put(4 * piece, lo[0], lo[1], lo[2], lo[3]);
        put(4 * piece + 1, lo[4], lo[5], lo[6], lo[7]);
        put(4 * piece + 2, hi[0], hi[1], hi[2], hi[3]);
        put(4 * piece + 3, hi[4], hi[5], hi[6], hi[7]);
      } else {
        const uint64_t dd = tc::f32x2(df, df), less = tc::f32x2(-8388736.f, -8388736.f);   // 2^23 + 128
        uint32_t x[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {   // bytes, 128 more, as the low bits of 2^23 (see s8_to_f32), two at a time
          const uint32_t u = w[i][j / 2] ^ 0x80808080u;
          const uint64_t n = tc::add_f32x2(tc::f32x2(__uint_as_float(__byte_perm(u, 0x4B000000u, 0x7540u | (2 * j % 4))),
                                                     __uint_as_float(__byte_perm(u, 0x4B000000u, 0x7540u | (2 * j % 4 + 1)))), less);
          float lo, hi;
          tc::f32x2_split(tc::mul_f32x2(n, dd), lo, hi);
          x[j] = tc::pack_bf16x2(lo, hi);
        }
        put(2 * piece, x[0], x[1], x[2], x[3]);
        put(2 * piece + 1, x[4], x[5], x[6], x[7]);
      }
    }
  }
};

}  // namespace fa
