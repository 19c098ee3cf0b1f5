// Writing and reading back a quantized K/V cache (fa_cache_write, fa_cache_read): the chunk's K and
// V go into the cached window that the attention entry points read in place (llama.cpp PR #57,
// commit 2394a4c). Both passes touch every byte once and are bound by HBM, or by their launch when
// a few rows are written, and writing many by its instructions. 67584 keys of 4 heads of 128 in 4 bits are read back to bf16 in
// 27 us, 6.5 TB/s, 96% of the measured copy rate, and written from it in 47 us, 3.8 TB/s (103 with a division for each
// feature; two lanes a block and one reciprocal leave less than half of the instructions); a token of 32 sequences with 8 heads is
// written in 2 us. Counters of the write of a whole window: issue 71% busy, ALU pipe 56%, DRAM 42%.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <type_traits>

#include "fa_check.h"
#include "fa_device.cuh"
#include "kv_pages.cuh"
#include "kv_quant.cuh"

namespace fa {
namespace {

__device__ __forceinline__ void load16(const float* p, float (&x)[16]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float4 a = __ldg(reinterpret_cast<const float4*>(p) + i);
    x[4 * i] = a.x; x[4 * i + 1] = a.y; x[4 * i + 2] = a.z; x[4 * i + 3] = a.w;
  }
}
__device__ __forceinline__ void load16(const __nv_bfloat16* p, float (&x)[16]) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint4 a = __ldg(reinterpret_cast<const uint4*>(p) + i);
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      x[8 * i + 2 * j] = __uint_as_float(w[j] << 16);
      x[8 * i + 2 * j + 1] = __uint_as_float(w[j] & 0xffff0000u);
    }
  }
}

// A thread quantizes 16 features of a row, two lanes a block of 32. blockIdx.y: 0 for K, 1 for V. Two rows a thread measured
// slower (58.4 us where this takes 47.0, see the head of the file), and lanes of 8 features, with twice the work for a block, 76.4.
// PAGED: the rows' places are found through the page table, each row's for itself.
template <typename T, int D, bool Q4, bool PAGED>
__global__ void __launch_bounds__(256) cache_write_kernel(CacheView c, PageView pages, RowView k, RowView v, unsigned rows,
                                                          unsigned n_rows, const int64_t* __restrict__ begin,
                                                          long long begin_all, const int64_t* __restrict__ count,
                                                          unsigned* status) {
  constexpr int LANES = D / 16;
  const unsigned g = blockIdx.x * (256 / LANES) + threadIdx.x / LANES;
  const int l = threadIdx.x % LANES;
  const RowView src = blockIdx.y ? v : k;
  float x[16];
#pragma unroll
  for (int j = 0; j < 16; ++j) x[j] = 0.f;
  bool on = false;
  size_t row = 0;
  if (g < rows) {
    const unsigned bh = g / n_rows, r = g % n_rows, b = bh / c.Hkv, h = bh % c.Hkv;
    const long long first = begin != nullptr ? __ldg(begin + b) : begin_all;
    if (count == nullptr || (long long)r < __ldg(count + b)) {
      if (first < c.S && first + r >= 0 && first + r < c.S) {
        on = true;
        if constexpr (PAGED) {
          const unsigned key = (unsigned)(first + r);
          const long long at = page_row(pages, c.Hkv, (int)b, (int)h, key & ~15u, l == 0 ? status : nullptr);
          on = at >= 0;
          row = (size_t)at + (key & 15u);
        } else {
          row = (size_t)bh * c.S + (size_t)(first + r);
        }
        if (on) load16(static_cast<const T*>(src.ptr) + b * src.sb + r * src.ss + h * src.sh + 16 * l, x);
      } else if (l == 0 && status != nullptr) {
        atomicCAS(status, 0u, 0x40000000u | kSiteCacheRow);
      }
    }
  }
  uint32_t w[4], p[2];
  const __half d = quantize_half_block<Q4>(x, w);
  const bool second = l & 1;
  if constexpr (Q4) {
    // features 16 .. 31 are the high four bits of features 0 .. 15; the first lane makes bytes 0 .. 7 of the block
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const uint32_t got = __shfl_xor_sync(0xffffffffu, second ? w[u] : w[2 + u], 1);
      p[u] = second ? got | w[2 + u] << 4 : w[u] | got << 4;
    }
  }
  if (!on) return;
  uint8_t* values = static_cast<uint8_t*>(blockIdx.y ? c.v_q : c.k_q);
  if constexpr (Q4) *reinterpret_cast<uint2*>(values + row * (D / 2) + 8 * l) = make_uint2(p[0], p[1]);
  else *reinterpret_cast<uint4*>(values + row * D + 16 * l) = make_uint4(w[0], w[1], w[2], w[3]);
  if (!second) (blockIdx.y ? c.v_d : c.k_d)[row * (D / 32) + l / 2] = __half_as_ushort(d);
}

// f(i, head, row, whether the head is another than the last time) for this thread's rows first, first + step, ...,
// without a division for each.
template <int ROWS, typename F>
__device__ __forceinline__ void each_row(unsigned first, unsigned step, unsigned rows, unsigned n_rows, F f) {
  unsigned bh = first / n_rows, r = first % n_rows;
  bool other = true;
#pragma unroll
  for (int i = 0; i < ROWS; ++i) {
    if (first + i * step >= rows) break;
    f(i, bh, r, other);
    r += step;
    other = r >= n_rows;
    if (other) {
      bh += r / n_rows;
      r %= n_rows;
    }
  }
}

// The values of a word of 4-bit numbers, pairs of neighbours: of its low nibbles to x, of its high ones to y. Masked, a
// nibble is an fp16 number, n 2^-24 or n 2^-20 (subnormal, exact); less 8 and times the scale, which has the power of two
// instead, it is exact in fp32. Half the instructions, on other pipes than the logic, of integers made floats one by one.
__device__ __forceinline__ void values_q4(uint32_t w, uint64_t d24, uint64_t d20, uint64_t* x, uint64_t* y) {
  const uint32_t h = w >> 8;
  auto less8 = [](uint32_t n, uint32_t off) {
    const __half2 r = __hadd2(*reinterpret_cast<const __half2*>(&n), *reinterpret_cast<const __half2*>(&off));
    return __half22float2(r);
  };
  const float2 e = less8(w & 0x000f000fu, 0x80088008u), o = less8(h & 0x000f000fu, 0x80088008u);   // bytes (0, 2), (1, 3)
  x[0] = tc::mul_f32x2(tc::f32x2(e.x, o.x), d24);
  x[1] = tc::mul_f32x2(tc::f32x2(e.y, o.y), d24);
  const float2 f = less8(w & 0x00f000f0u, 0x80808080u), p = less8(h & 0x00f000f0u, 0x80808080u);
  y[0] = tc::mul_f32x2(tc::f32x2(f.x, p.x), d20);
  y[1] = tc::mul_f32x2(tc::f32x2(f.y, p.y), d20);
}

// 16 bytes of values.
__device__ __forceinline__ void store16(float* p, const uint64_t (&x)[2]) {
  float4 v;
  tc::f32x2_split(x[0], v.x, v.y);
  tc::f32x2_split(x[1], v.z, v.w);
  *reinterpret_cast<float4*>(p) = v;
}
__device__ __forceinline__ void store16(__nv_bfloat16* p, const uint64_t (&x)[4]) {
  uint32_t u[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float lo, hi;
    tc::f32x2_split(x[i], lo, hi);
    u[i] = tc::pack_bf16x2(lo, hi);
  }
  *reinterpret_cast<uint4*>(p) = make_uint4(u[0], u[1], u[2], u[3]);
}

// A thread reads N bytes of numbers of ROWS rows, all of them on their way at once, and writes N features of 16 bytes, which
// with its neighbours' fill whole sectors (q4_0: two times N, of the low and of the high nibbles). blockIdx.y: 0 for K, 1 for V.
// PLACED: rows are found through a page table, or from a begin of each sequence's own, or both; one that the cache does not
// have is read as zeros.
template <typename T, int D, bool Q4, int ROWS, bool PLACED>
__global__ void __launch_bounds__(256) cache_read_kernel(CacheView c, PageView pages, const int64_t* __restrict__ begins,
                                                         long long begin, unsigned rows, unsigned n_rows, RowView k,
                                                         RowView v, unsigned* status) {
  constexpr int N = 16 / sizeof(T), PARTS = (Q4 ? D / 2 : D) / N, STEP = 256 / PARTS;   // rows a block takes at a time
  const int part = threadIdx.x % PARTS;
  const unsigned first = blockIdx.x * (STEP * ROWS) + threadIdx.x / PARTS;
  const RowView dst = blockIdx.y ? v : k;
  const uint8_t* values = static_cast<const uint8_t*>(blockIdx.y ? c.v_q : c.k_q) + N * part;
  const int blk = N * part / (Q4 ? 16 : 32);
  const uint16_t* scales = (blockIdx.y ? c.v_d : c.k_d) + blk;
  uint32_t w[ROWS][N / 4];
  uint16_t scale[ROWS];
  each_row<ROWS>(first, STEP, rows, n_rows, [&](int i, unsigned bh, unsigned r, bool) {
    size_t row = (size_t)bh * c.S + (size_t)(begin + r);
    if constexpr (PLACED) {
      const unsigned b = bh / c.Hkv, h = bh % c.Hkv;
      const long long from = begins != nullptr ? __ldg(begins + b) : begin;
      const bool inside = from < c.S && from + r >= 0 && from + r < c.S;
      if (!inside && part == 0 && status != nullptr) atomicCAS(status, 0u, 0x40000000u | kSiteCacheRow);
      const unsigned key = inside ? (unsigned)(from + r) : 0u;
      long long at = inside ? (long long)bh * c.S + key : -1;
      if (inside && pages.table != nullptr) {
        at = page_row(pages, c.Hkv, (int)b, (int)h, key & ~15u, part == 0 ? status : nullptr);
        if (at >= 0) at += key & 15u;
      }
      scale[i] = 0;
#pragma unroll
      for (int j = 0; j < N / 4; ++j) w[i][j] = Q4 ? 0x88888888u : 0u;
      if (at < 0) return;
      row = (size_t)at;
    }
    scale[i] = __ldg(scales + row * (D / 32));
    const uint8_t* at = values + row * (Q4 ? D / 2 : D);
    if constexpr (N == 8) {
      const uint2 u = __ldg(reinterpret_cast<const uint2*>(at));
      w[i][0] = u.x;
      w[i][1] = u.y;
    } else {
      w[i][0] = __ldg(reinterpret_cast<const uint32_t*>(at));
    }
  });
  T* head = nullptr;
  each_row<ROWS>(first, STEP, rows, n_rows, [&](int i, unsigned bh, unsigned r, bool other) {
    if (other) head = static_cast<T*>(dst.ptr) + bh / c.Hkv * dst.sb + bh % c.Hkv * dst.sh + (Q4 ? blk * 32 + N * part % 16 : N * part);
    const float d = __half2float(__ushort_as_half(scale[i]));
    T* out = head + r * dst.ss;
    uint64_t x[N / 2];
    if constexpr (Q4) {
      const uint64_t d24 = tc::f32x2(d * 16777216.f, d * 16777216.f), d20 = tc::f32x2(d * 1048576.f, d * 1048576.f);
      uint64_t y[N / 2];
#pragma unroll
      for (int j = 0; j < N / 4; ++j) values_q4(w[i][j], d24, d20, x + 2 * j, y + 2 * j);
      store16(out, x);
      store16(out + 16, y);
    } else {
      const uint64_t dd = tc::f32x2(d, d);
#pragma unroll
      for (int j = 0; j < N / 2; ++j) {
        const uint32_t u = w[i][j / 2] ^ 0x80808080u;
        x[j] = tc::mul_f32x2(tc::f32x2(s8_to_f32(u, 2 * j % 4), s8_to_f32(u, 2 * j % 4 + 1)), dd);
      }
      store16(out, x);
    }
  });
}

constexpr long long kMaxRows = 0x7fffffffLL;   // the kernels count rows in 32 bits

// Blocks that take `per_block` rows each; 0 when the rows are too many.
unsigned blocks_for(long long rows, int per_block) {
  return rows > kMaxRows ? 0u : (unsigned)((rows + per_block - 1) / per_block);
}

}  // namespace

cudaError_t launch_cache_write(const CacheView& c, const PageView& pages, const RowView& k, const RowView& v, int dtype,
                               int n_rows, const int64_t* begin, long long begin_all, const int64_t* count,
                               unsigned* status, cudaStream_t st) {
  const long long rows = (long long)c.B * c.Hkv * n_rows;
  const unsigned n = blocks_for(rows, 256 / (c.D / 16));
  if (n == 0) return cudaErrorInvalidConfiguration;
  auto go = [&](auto kernel) {
    kernel<<<dim3(n, 2), 256, 0, st>>>(c, pages, k, v, (unsigned)rows, (unsigned)n_rows, begin, begin_all, count, status);
  };
  const bool paged = pages.table != nullptr;
  auto by_format = [&](auto t, auto dim) {
    using T = decltype(t);
    constexpr int D = decltype(dim)::value;
    if (c.q4) paged ? go(cache_write_kernel<T, D, true, true>) : go(cache_write_kernel<T, D, true, false>);
    else paged ? go(cache_write_kernel<T, D, false, true>) : go(cache_write_kernel<T, D, false, false>);
  };
  using D64 = std::integral_constant<int, 64>;
  using D128 = std::integral_constant<int, 128>;
  if (dtype == DT_BF16) c.D == 64 ? by_format(__nv_bfloat16{}, D64{}) : by_format(__nv_bfloat16{}, D128{});
  else c.D == 64 ? by_format(float{}, D64{}) : by_format(float{}, D128{});
  count_launches(1);
  return cudaGetLastError();
}

namespace {

template <bool PLACED>
cudaError_t read_rows(const CacheView& c, const PageView& pages, const int64_t* begins, long long begin, int n_rows, int dtype,
                      const RowView& k, const RowView& v, unsigned* status, cudaStream_t st) {
  const long long rows = (long long)c.B * c.Hkv * n_rows;
  const int parts = (c.q4 ? c.D / 2 : c.D) / (dtype == DT_BF16 ? 8 : 4), step = 256 / parts;
  // four rows a thread, where that still leaves blocks for every SM (67584 keys of 4 heads in 4 bits: 27.2 us; one 31.6, eight 27.4)
  const bool many = rows >= 8LL * step * sm_count();
  const unsigned n = blocks_for(rows, many ? 4 * step : step);
  if (n == 0) return cudaErrorInvalidConfiguration;
  auto go = [&](auto kernel) {
    kernel<<<dim3(n, 2), 256, 0, st>>>(c, pages, begins, begin, (unsigned)rows, (unsigned)n_rows, k, v, status);
  };
  auto by_format = [&](auto t, auto dim) {
    using T = decltype(t);
    constexpr int D = decltype(dim)::value;
    if (c.q4) many ? go(cache_read_kernel<T, D, true, 4, PLACED>) : go(cache_read_kernel<T, D, true, 1, PLACED>);
    else many ? go(cache_read_kernel<T, D, false, 4, PLACED>) : go(cache_read_kernel<T, D, false, 1, PLACED>);
  };
  using D64 = std::integral_constant<int, 64>;
  using D128 = std::integral_constant<int, 128>;
  if (dtype == DT_BF16) c.D == 64 ? by_format(__nv_bfloat16{}, D64{}) : by_format(__nv_bfloat16{}, D128{});
  else c.D == 64 ? by_format(float{}, D64{}) : by_format(float{}, D128{});
  count_launches(1);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_cache_read(const CacheView& c, long long begin, int n_rows, int dtype, const RowView& k,
                              const RowView& v, cudaStream_t st) {
  return read_rows<false>(c, PageView{}, nullptr, begin, n_rows, dtype, k, v, nullptr, st);
}

namespace {

fa_status check_planes(const fa_cache* c, bool pool, CacheView& out) {
  if (c == nullptr) { set_error("cache is NULL"); return FA_ERR_INVALID_ARG; }
  if (c->B < 1 || (c->B > 65535 && !pool) || c->Hkv < 1 || c->Hkv > 65535) {
    set_error("cache B=%d, Hkv=%d: each in [1, 65535]", c->B, c->Hkv); return FA_ERR_INVALID_ARG;
  }
  if (c->S < 1 || c->S > kMaxSeq) { set_error("cache S=%d outside [1, %d]", c->S, kMaxSeq); return FA_ERR_INVALID_ARG; }
  if (c->D <= 0) { set_error("D=%d must be positive", c->D); return FA_ERR_INVALID_ARG; }
  if (c->D != 64 && c->D != 128) { set_error("D=%d unsupported (64 or 128)", c->D); return FA_ERR_UNSUPPORTED; }
  if (c->kv_format != FA_KV_Q8_0 && c->kv_format != FA_KV_Q4_0) {
    set_error("cache kv_format=%d: FA_KV_Q8_0 or FA_KV_Q4_0", c->kv_format); return FA_ERR_INVALID_ARG;
  }
  if (c->reserved != 0) { set_error("reserved field must be 0"); return FA_ERR_INVALID_ARG; }
  if (too_large(c->B, c->Hkv, c->S, c->D)) {
    set_error("a cache of these shapes would hold more than 2^40 elements"); return FA_ERR_INVALID_ARG;
  }
  out = CacheView{c->B, c->Hkv, c->S, c->D, c->kv_format == FA_KV_Q4_0, c->k_q, c->k_d, c->v_q, c->v_d};
  return FA_OK;
}

}  // namespace

fa_status check_cache(const fa_cache* c, CacheView& out) { return check_planes(c, false, out); }

fa_status check_paged(const fa_cache* c, const fa_pages* pages, CacheView& held, CacheView& seen, PageView& view, Span& table) {
  const fa_status st = check_planes(c, pages != nullptr, held);
  if (st != FA_OK) return st;
  seen = held;
  view = PageView{};
  table = Span{nullptr, 0, "table"};
  if (pages == nullptr) return FA_OK;
  if (pages->B < 1 || pages->B > 65535) { set_error("pages B=%d outside [1, 65535]", pages->B); return FA_ERR_INVALID_ARG; }
  if (held.S % 16 != 0) { set_error("pages of %d keys: a multiple of 16", held.S); return FA_ERR_INVALID_ARG; }
  if (pages->M < 1 || (long long)pages->M * held.S > kMaxSeq) {
    set_error("%d pages of %d keys a sequence: 1 to %d keys", pages->M, held.S, kMaxSeq); return FA_ERR_INVALID_ARG;
  }
  if (pages->table == nullptr || (uintptr_t)pages->table % 4 != 0) {
    set_error("table is NULL or not 4-byte aligned"); return FA_ERR_INVALID_ARG;
  }
  if (pages->B > 1 && (pages->stride < pages->M || (double)pages->stride * pages->B > kMaxElems)) {
    set_error("table stride of %lld: at least its %d pages, and at most 2^40 elements in all", (long long)pages->stride, pages->M);
    return FA_ERR_INVALID_ARG;
  }
  seen.B = pages->B;
  seen.S = pages->M * held.S;
  if (too_large(seen.B, seen.Hkv, seen.S, seen.D)) {
    set_error("the sequences' keys would be more than 2^40 elements"); return FA_ERR_INVALID_ARG;
  }
  const unsigned long long units = (unsigned)held.S / 16;
  view = PageView{pages->table, pages->B > 1 ? (long long)pages->stride : 0, ((1ull << 40) + units - 1) / units, (unsigned)held.S,
                  (unsigned)held.B};
  table.p = pages->table;
  table.n = ((size_t)view.stride * (pages->B - 1) + pages->M) * 4;
  return FA_OK;
}

void cache_spans(const CacheView& c, Span out[4]) {
  const size_t n = (size_t)c.B * c.Hkv * c.S * c.D;
  out[0] = {c.k_q, c.q4 ? n / 2 : n, "k_q"};
  out[1] = {c.k_d, n / 16, "k_d"};   // one fp16 for 32 features
  out[2] = {c.v_q, c.q4 ? n / 2 : n, "v_q"};
  out[3] = {c.v_d, n / 16, "v_d"};
}

namespace {

fa_status check_rows(const CacheView& c, const fa_view* k, const fa_view* v, int dtype, int n_rows, bool written,
                     Span out[2]) {
  if (dtype != FA_F32 && dtype != FA_BF16) { set_error("dtype=%d invalid", dtype); return FA_ERR_INVALID_ARG; }
  if (n_rows < 0 || n_rows > kMaxSeq) { set_error("n_rows=%d outside [0, %d]", n_rows, kMaxSeq); return FA_ERR_INVALID_ARG; }
  if (too_large(c.B, c.Hkv, n_rows, c.D)) {
    set_error("K or V would hold more than 2^40 elements"); return FA_ERR_INVALID_ARG;
  }
  if ((long long)c.B * c.Hkv * n_rows > kMaxRows) { set_error("too many rows for one launch"); return FA_ERR_UNSUPPORTED; }
  const size_t es = dtype == FA_BF16 ? 2 : 4;
  fa_status st = check_view(k, c.B, n_rows, c.Hkv, c.D, es, written, "k", out[0]);
  return st != FA_OK ? st : check_view(v, c.B, n_rows, c.Hkv, c.D, es, written, "v", out[1]);
}

}  // namespace
}  // namespace fa

using namespace fa;

extern "C" {

fa_status fa_cache_write_pages(const fa_cache* c, const fa_pages* pages, const fa_view* k, const fa_view* v, int32_t dtype,
                               int32_t n_rows, const int64_t* begin, int64_t begin_all, const int64_t* count, void* stream) {
  clear_error();
  CacheView held, cv;
  PageView pv;
  Span in[5], out[4];
  fa_status st = check_paged(c, pages, held, cv, pv, in[4]);
  if (st != FA_OK) return st;
  if ((st = check_rows(cv, k, v, dtype, n_rows, false, in)) != FA_OK) return st;
  if (begin == nullptr && (begin_all < 0 || begin_all > cv.S - n_rows)) {
    set_error("rows [%lld, +%d) outside the %d keys", (long long)begin_all, n_rows, cv.S); return FA_ERR_INVALID_ARG;
  }
  if ((uintptr_t)begin % 8 != 0 || (uintptr_t)count % 8 != 0) {
    set_error("begin and count must be 8-byte aligned"); return FA_ERR_INVALID_ARG;
  }
  if (n_rows == 0) return FA_OK;
  cache_spans(held, out);
  if ((st = check_buffers(in, 2, out, 4)) != FA_OK) return st;
  in[2] = {begin, begin != nullptr ? (size_t)cv.B * 8 : 0, "begin"};
  in[3] = {count, count != nullptr ? (size_t)cv.B * 8 : 0, "count"};
  if ((st = check_apart(in + 2, 3, out, 4)) != FA_OK) return st;
  return cuda_status(launch_cache_write(cv, pv, row_view(k), row_view(v), dtype, n_rows, begin, begin_all, count,
                                        device_status_ptr(), (cudaStream_t)stream),
                     "cache write launch");
}

fa_status fa_cache_write(const fa_cache* c, const fa_view* k, const fa_view* v, int32_t dtype, int32_t n_rows,
                         const int64_t* begin, int64_t begin_all, const int64_t* count, void* stream) {
  return fa_cache_write_pages(c, nullptr, k, v, dtype, n_rows, begin, begin_all, count, stream);
}

fa_status fa_cache_read_pages(const fa_cache* c, const fa_pages* pages, const int64_t* begins, int64_t begin, int32_t n_rows,
                              int32_t dtype, const fa_view* k, const fa_view* v, void* stream) {
  clear_error();
  CacheView held, cv;
  PageView pv;
  Span in[6], out[2];
  fa_status st = check_paged(c, pages, held, cv, pv, in[4]);
  if (st != FA_OK) return st;
  if ((st = check_rows(cv, k, v, dtype, n_rows, true, out)) != FA_OK) return st;
  if (begins == nullptr && (begin < 0 || begin > cv.S - n_rows)) {
    set_error("rows [%lld, +%d) outside the %d keys", (long long)begin, n_rows, cv.S); return FA_ERR_INVALID_ARG;
  }
  if ((uintptr_t)begins % 8 != 0) { set_error("begin must be 8-byte aligned"); return FA_ERR_INVALID_ARG; }
  if (n_rows == 0) return FA_OK;
  cache_spans(held, in);
  const size_t es = dtype == FA_BF16 ? 2 : 4;
  if ((st = check_buffers(in, 4, out, 2, side_by_side(k, cv.Hkv, v, cv.Hkv, cv.B, n_rows, cv.D, es))) != FA_OK) return st;
  in[5] = {begins, begins != nullptr ? (size_t)cv.B * 8 : 0, "begin"};
  if ((st = check_apart(in + 4, 2, out, 2)) != FA_OK) return st;
  const RowView kr = row_view(k), vr = row_view(v);
  const cudaStream_t cs = (cudaStream_t)stream;
  const cudaError_t e = pages == nullptr && begins == nullptr
                            ? launch_cache_read(cv, begin, n_rows, dtype, kr, vr, cs)
                            : read_rows<true>(cv, pv, begins, begin, n_rows, dtype, kr, vr, device_status_ptr(), cs);
  return cuda_status(e, "cache read launch");
}

fa_status fa_cache_read(const fa_cache* c, int64_t begin, int32_t n_rows, int32_t dtype, const fa_view* k,
                        const fa_view* v, void* stream) {
  return fa_cache_read_pages(c, nullptr, nullptr, begin, n_rows, dtype, k, v, stream);
}

}  // extern "C"
