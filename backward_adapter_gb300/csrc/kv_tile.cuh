// A tile of 128 keys of a quantized plane as the bf16 operand of tcgen05.mma: four warps read 32 rows each, 16 bytes a lane
// and load, and write them in the 128-byte-swizzled layout that TMA would have written (64-feature boxes of 128 rows x 128
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

// What a warp reads for its rows 32 w .. 32 w + 31 of a tile: where the two runs of 16 rows begin in a plane (-1: no page),
// and how many of the 32 keys there are.
struct TileRows {
  long long row0, row1;
  int keys;
};

// Of sequence b's head h, keys key0 .. key0 + 31, `len` keys in all.
template <bool PAGED>
__device__ __forceinline__ TileRows tile_rows(const CacheView& c, const PageView& pages, int b, int h, int key0, int len,
                                              unsigned* status) {
  TileRows t;
  t.keys = min(max(len - key0, 0), 32);
  if constexpr (PAGED) {
    t.row0 = t.keys > 0 ? page_row(pages, c.Hkv, b, h, key0, status) : -1;
    t.row1 = t.keys > 16 ? page_row(pages, c.Hkv, b, h, key0 + 16, status) : -1;
  } else {
    t.row0 = ((long long)b * c.Hkv + h) * c.S + key0;
    t.row1 = t.row0 + 16;
  }
  return t;
}

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

// The bytes of a warp's rows, in registers.
template <int D, bool Q4>
struct TileBytes {
  static constexpr int ROW = Q4 ? D / 2 : D;   // bytes of a row
  static constexpr int N = ROW / 16;           // pieces of 16 bytes in a row, and loads of a lane
  static constexpr int BOX = 128 * 128;        // bytes of a 64-feature box of the tile
  uint32_t w[N][4];
  uint16_t d[N];

  // Load i: the lane's row among the 32, and which piece of it.
  __device__ static __forceinline__ int row_of(int i, int lane) {
    return N == 2 ? 16 * i + 8 * (lane >> 4) + (lane & 7) : N == 4 ? 8 * i + (lane & 7) : 8 * (i >> 1) + (lane & 7);
  }
  __device__ static __forceinline__ int piece_of(int i, int lane) {
    return N == 2 ? (lane >> 3) & 1 : N == 4 ? lane >> 3 : 4 * (i & 1) + (lane >> 3);
  }

  // Kept in this place among the waits; rows that are not there are zeros, and not read.
  __device__ __forceinline__ void load(const void* values, const uint16_t* scales, const TileRows& t) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int row = row_of(i, lane), piece = piece_of(i, lane);
      const long long first = (i < N / 2 ? t.row0 : t.row1 - 16);   // of the second run as if the first had been before it
      const bool on = row < t.keys && (i < N / 2 ? t.row0 : t.row1) >= 0;
      w[i][0] = w[i][1] = w[i][2] = w[i][3] = Q4 ? 0x88888888u : 0u;
      d[i] = 0;
      if (on) {
        const uint8_t* src = static_cast<const uint8_t*>(values) + (first + row) * ROW + 16 * piece;
        asm volatile("ld.global.nc.v4.b32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(w[i][0]), "=r"(w[i][1]), "=r"(w[i][2]), "=r"(w[i][3]) : "l"(src));
        asm volatile("ld.global.nc.u16 %0, [%1];" : "=h"(d[i]) : "l"(scales + (first + row) * (D / 32) + (Q4 ? piece : piece / 2)));
      }
    }
  }

  // Into rows 32 w .. of the tile at `tile` (shared memory). FINITE: a scale that is not finite counts as 0.
  template <bool FINITE>
  __device__ __forceinline__ void store(uint32_t tile, int warp) const {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int piece = piece_of(i, lane);
      float df = __half2float(__ushort_as_half(d[i]));
      if (FINITE && !(fabsf(df) <= 65504.f)) df = 0.f;
      const uint32_t at = tile + (32 * warp + row_of(i, lane)) * 128;
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
        const uint64_t dd = tc::f32x2(df, df);
        uint32_t x[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const uint32_t u = w[i][j / 2] ^ 0x80808080u;
          float lo, hi;
          tc::f32x2_split(tc::mul_f32x2(tc::f32x2(s8_to_f32(u, 2 * j % 4), s8_to_f32(u, 2 * j % 4 + 1)), dd), lo, hi);
          x[j] = tc::pack_bf16x2(lo, hi);
        }
        put(2 * piece, x[0], x[1], x[2], x[3]);
        put(2 * piece + 1, x[4], x[5], x[6], x[7]);
      }
    }
  }
};

}  // namespace fa
