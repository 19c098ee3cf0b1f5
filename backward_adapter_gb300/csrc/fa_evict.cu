// Eviction from a quantized cache by accumulated attention weight (fa_cache_evict): of each head's keys the ones that matter
// are found and moved together.
//
// A cluster of blocks has one head of one sequence, a run of its keys for each block. The border between what stays and what
// goes is found a digit of 8 bits at a time, the highest first: every block counts its keys' digits, the counts are added
// over the cluster through its shared memory, and the digit in which the wanted number is reached is the border's. Keys
// above the border stay, and the first of those at it: with the counts of both in the blocks and threads before, every key knows
// its new place, and writes its index there (kept).
//
// Moved is in waves where places and sources may be the same memory (the rows of the same pages, the weights in place): a
// wave of places is loaded by the whole cluster before any of it is stored; a key never moves up, so a wave's places hold none
// of a later wave's keys. Rows that go to other pages are a kernel's of their own, all rows at once: the heads of one sequence
// do not fill the machine, and there is nothing to wait for.
//
// Measured (device time), D = 128: 64 sequences of 1024 to 8192 keys, 8 heads, in 4 bits, cut to 2048 keys in other pages: 91 us, of
// which the rows are 61, 4.9 TB/s of reading and writing, 74% of the measured copy rate, and finding them 30 (instructions: each
// key is looked at six times, in shared memory). One sequence of 67,584 keys, 4 heads, in 8 bits, cut to 8448: 34 us with what
// was kept read back; finding is 21 of it, 64 blocks that wait for each other six times. In place, where a wave waits for its loads and
// one head's blocks move its rows, the batch takes 112 us in pages and 101 in one piece, the window 40 and 34 (25 to other pages, without
// what is read back).
#include <cuda_runtime.h>

#include <type_traits>

#include "fa_check.h"
#include "fa_device.cuh"
#include "kv_pages.cuh"
#include "tc_ptx.cuh"

namespace fa {
namespace {

constexpr int kThreads = 512;
constexpr int kCluster = 16;       // blocks of a head, at most (four heads of 67,584 keys: 42.6 us with 8, 38.0 with 16)
constexpr int kCached = 10240;     // keys whose weights a block holds in shared memory, within 48 KB; more are read again
constexpr int kEach = 4;           // keys a thread looks at in turn
constexpr int kStep = kThreads * kEach;

struct EvictArgs {
  CacheView c;
  PageView from, to;
  const float* weights;
  const int64_t* lengths;
  float* weights_out;
  int32_t* kept;
  int64_t* new_lengths;
  unsigned* status;
  long long W;
  int keep, sinks, recent;
  int cached;
};

__device__ __forceinline__ unsigned cluster_rank() {
  unsigned r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ unsigned cluster_size() {
  unsigned r;
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
  return r;
}
// What the cluster's threads wrote before, to shared or global memory, is there for all of them after.
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
}
// ... of one block's threads where it is a cluster by itself, without what makes global memory the others'.
__device__ __forceinline__ void sync_all(unsigned blocks) {
  if (blocks == 1) __syncthreads();
  else cluster_sync();
}
__device__ __forceinline__ unsigned read_of(unsigned rank, const unsigned* p) {
  unsigned at, v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(tc::smem_u32(p)), "r"(rank));
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(at) : "memory");
  return v;
}

// Weights as whole numbers in the same order; no number is the least, and -0 is 0.
__device__ __forceinline__ unsigned ordered(float w) {
  if (w != w) return 0u;
  const unsigned u = w == 0.f ? 0u : __float_as_uint(w);
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}

// Exclusive sum of x over the block's threads, and of all; `sums` has a word for each warp.
__device__ __forceinline__ unsigned block_sum_before(unsigned x, unsigned* sums, unsigned& all) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  unsigned y = x;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const unsigned z = __shfl_up_sync(0xffffffffu, y, o);
    if (lane >= o) y += z;
  }
  __syncthreads();   // the last call's sums are read
  if (lane == 31) sums[warp] = y;
  __syncthreads();
  unsigned before = y - x;
  all = 0;
#pragma unroll
  for (int w = 0; w < kThreads / 32; ++w) {
    const unsigned s = sums[w];
    if (w < warp) before += s;
    all += s;
  }
  return before;
}

// Row of the planes that holds key j of head h of sequence b: -1 where the table names no page.
template <bool PAGED>
__device__ __forceinline__ long long place_of(const EvictArgs& a, const PageView& pages, unsigned bh, int b, int h, int j) {
  if constexpr (!PAGED) return (long long)bh * a.c.S + j;
  const long long row = page_row(pages, a.c.Hkv, b, h, j & ~15, a.status);
  return row < 0 ? -1 : row + (j & 15);
}

// A thread's part of a key's row: 16 bytes of the numbers of K or of V, with the first ones their scales.
template <int D, bool Q4>
struct RowParts {
  static constexpr int ROW = Q4 ? D / 2 : D, PIECES = ROW / 16, LANES = 2 * PIECES, NB = D / 32;
  using Scales = std::conditional_t<NB == 4, uint2, uint32_t>;
  struct Data { uint4 x; Scales d; };
  uint8_t* values;
  uint16_t* scales;
  bool first;
  __device__ __forceinline__ RowParts(const CacheView& c, int lane) {
    const bool v = lane >= PIECES;
    first = lane % PIECES == 0;
    values = static_cast<uint8_t*>(v ? c.v_q : c.k_q) + 16 * (lane % PIECES);
    scales = v ? c.v_d : c.k_d;
  }
  __device__ __forceinline__ Data load(long long row) const {   // of no row: zeros
    const uint32_t zero = Q4 ? 0x88888888u : 0u;
    Data r{make_uint4(zero, zero, zero, zero), Scales{}};
    if (row >= 0) {
      r.x = *reinterpret_cast<const uint4*>(values + row * ROW);
      if (first) r.d = *reinterpret_cast<const Scales*>(scales + row * NB);
    }
    return r;
  }
  __device__ __forceinline__ void store(long long row, const Data& r) const {
    *reinterpret_cast<uint4*>(values + row * ROW) = r.x;
    if (first) *reinterpret_cast<Scales*>(scales + row * NB) = r.d;
  }
};

// MOVE: the rows too, in place.
template <int D, bool Q4, bool PAGED, bool MOVE>
__global__ void __launch_bounds__(kThreads) evict_kernel(const __grid_constant__ EvictArgs a) {
  extern __shared__ unsigned cache[];   // [cached]: the order of this block's first keys
  __shared__ unsigned counts[4][256], total[256], sums[kThreads / 32], found[2], own[2];
  const unsigned rank = cluster_rank(), blocks = cluster_size();
  const unsigned bh = blockIdx.x / blocks;
  const int b = bh / a.c.Hkv, h = bh % a.c.Hkv;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;

  let_next_kernel_start();
  const long long length = __ldg(a.lengths + b);
  const int len = (int)min(max(length, 0LL), min((long long)a.c.S, a.W));
  const int left = min(len, a.keep);
  if (rank == 0 && h == 0 && threadIdx.x == 0) {
    if (len != length && a.status != nullptr) atomicCAS(a.status, 0u, 0x40000000u | kSiteDecodeLength);
    a.new_lengths[b] = left;
  }
  const float* weights = a.weights + (size_t)bh * a.W;
  float* weights_out = a.weights_out + (size_t)bh * a.W;
  int32_t* kept = a.kept + (size_t)bh * a.keep;
  const int all_threads = blocks * kThreads, me = rank * kThreads + threadIdx.x;

  if (len <= a.keep) {
    for (int i = me; i < a.keep; i += all_threads) kept[i] = i < len ? i : -1;
  } else {
    // the sinks and the last ones; between them this block's keys [first, first + n)
    for (int i = me; i < a.sinks; i += all_threads) kept[i] = i;
    for (int i = me; i < a.recent; i += all_threads) kept[a.keep - a.recent + i] = len - a.recent + i;
    const int middle = len - a.sinks - a.recent, per = (middle + blocks - 1) / blocks;
    const int first = min((int)rank * per, middle), n = min(per, middle - first);
    const float* w = weights + a.sinks + first;
    for (int i = threadIdx.x; i < min(n, a.cached); i += kThreads) cache[i] = ordered(w[i]);
    for (int i = threadIdx.x; i < 4 * 256; i += kThreads) counts[i / 256][i % 256] = 0;
    __syncthreads();
    auto key = [&](int i) { return i < a.cached ? cache[i] : ordered(w[i]); };

    unsigned border = 0xffffffffu, at_border = 0;   // above every weight: nothing is wanted
    unsigned wanted = a.keep - a.sinks - a.recent;
    if (wanted > 0) {
      border = 0;
#pragma unroll 1
      for (int pass = 0; pass < 4; ++pass) {
        const int shift = 24 - 8 * pass;
        // one add for each key, as many lanes of a warp as may have its digit: 21.0 us for 256 heads of 8192 keys whose weights are
        // spread over 2^57 or all 0; lanes that agree with the first counted together first, 26.8 and 31.1
        for (int i = threadIdx.x; i < n; i += kThreads) {
          const unsigned u = key(i);
          if (pass == 0 || (u ^ border) >> (shift + 8) == 0) atomicAdd(&counts[pass][u >> shift & 255u], 1u);
        }
        sync_all(blocks);
        if (blocks == 1) {
          if (threadIdx.x < 256) total[threadIdx.x] = counts[pass][threadIdx.x];
        } else if (threadIdx.x < 256) {
          unsigned x[kCluster], sum = 0;   // all on their way at once
#pragma unroll
          for (unsigned r = 0; r < kCluster; ++r) x[r] = r < blocks ? read_of(r, &counts[pass][threadIdx.x]) : 0u;
#pragma unroll
          for (unsigned r = 0; r < kCluster; ++r) sum += x[r];
          total[threadIdx.x] = sum;
        }
        __syncthreads();
        if (warp == 0) {   // lane l has the digits 255 - 8 l and the seven below
          unsigned x = 0;
#pragma unroll
          for (int k = 0; k < 8; ++k) x += total[255 - 8 * lane - k];
          unsigned y = x;
#pragma unroll
          for (int o = 1; o < 32; o <<= 1) {
            const unsigned z = __shfl_up_sync(0xffffffffu, y, o);
            if (lane >= o) y += z;
          }
          if (y >= wanted && y - x < wanted) {   // one lane
            unsigned rest = wanted - (y - x);
            int digit = 255 - 8 * lane;
            while (total[digit] < rest) rest -= total[digit--];
            found[0] = border | (unsigned)digit << shift;
            found[1] = rest;
          }
        }
        __syncthreads();
        border = found[0];
        wanted = found[1];
      }
      at_border = wanted;
    }

    // keys above and at the border, of the blocks before and of the threads before
    unsigned above = 0, equal = 0;
    for (int i = threadIdx.x; i < n; i += kThreads) {
      const unsigned u = key(i);
      above += u > border;
      equal += u == border;
    }
    unsigned all_above, all_equal;
    block_sum_before(above, sums, all_above);
    block_sum_before(equal, sums, all_equal);
    if (threadIdx.x == 0) {
      own[0] = all_above;
      own[1] = all_equal;
    }
    sync_all(blocks);
    // lane r reads what block r has
    unsigned above_before = (unsigned)lane < rank ? read_of(lane, &own[0]) : 0u, equal_before = (unsigned)lane < rank ? read_of(lane, &own[1]) : 0u;
#pragma unroll
    for (int o = kCluster / 2; o > 0; o >>= 1) {
      above_before += __shfl_xor_sync(0xffffffffu, above_before, o);
      equal_before += __shfl_xor_sync(0xffffffffu, equal_before, o);
    }
    above_before = __shfl_sync(0xffffffffu, above_before, 0);
    equal_before = __shfl_sync(0xffffffffu, equal_before, 0);
    for (int i0 = 0; i0 < n; i0 += kStep) {
      const int i1 = i0 + threadIdx.x * kEach;
      unsigned u[kEach], x = 0;
#pragma unroll
      for (int k = 0; k < kEach; ++k) {
        u[k] = i1 + k < n ? key(i1 + k) : 0u;
        if (i1 + k < n) x += u[k] > border ? 1u << 16 : u[k] == border ? 1u : 0u;
      }
      unsigned all;
      const unsigned before = block_sum_before(x, sums, all);
      unsigned g = above_before + (before >> 16), e = equal_before + (before & 0xffffu);
#pragma unroll
      for (int k = 0; k < kEach; ++k) {
        if (i1 + k >= n) break;
        const bool more = u[k] > border, same = u[k] == border;
        if (more || (same && e < at_border)) kept[a.sinks + g + min(e, at_border)] = a.sinks + first + i1 + k;
        g += more;
        e += same;
      }
      above_before += all >> 16;
      equal_before += all & 0xffffu;
    }
  }
  sync_all(blocks);   // kept is there

  if constexpr (MOVE) {   // the rows: a thread has 16 bytes of K's or V's numbers, the first one of a row its scales too
    using R = RowParts<D, Q4>;
    constexpr int PER = kThreads / R::LANES, AHEAD = 4;   // rows of a block at a time, and on their way
    const R part(a.c, threadIdx.x % R::LANES);
    const int wave = PER * AHEAD * blocks;
    for (int i0 = 0; i0 < left; i0 += wave) {
      typename R::Data x[AHEAD];
      long long to[AHEAD];
#pragma unroll
      for (int k = 0; k < AHEAD; ++k) {
        const int i = i0 + (k * blocks + rank) * PER + threadIdx.x / R::LANES;
        to[k] = -1;
        if (i >= left) continue;
        const int j = kept[i];
        if (j == i) continue;   // it stays where it is
        to[k] = place_of<PAGED>(a, a.to, bh, b, h, i);
        x[k] = part.load(place_of<PAGED>(a, a.from, bh, b, h, j));
      }
      sync_all(blocks);   // all of the wave is read
#pragma unroll
      for (int k = 0; k < AHEAD; ++k)
        if (to[k] >= 0) part.store(to[k], x[k]);
    }
  }
  constexpr int SOME = 4;   // the weights: four of a thread at a time
  for (int i0 = 0; i0 < left; i0 += SOME * all_threads) {
    float x[SOME];
#pragma unroll
    for (int k = 0; k < SOME; ++k) {
      const int i = i0 + k * all_threads + me;
      if (i < left) x[k] = weights[kept[i]];
    }
    sync_all(blocks);
#pragma unroll
    for (int k = 0; k < SOME; ++k) {
      const int i = i0 + k * all_threads + me;
      if (i < left) weights_out[i] = x[k];
    }
  }
  for (long long i = left + me; i < a.W; i += all_threads) weights_out[i] = 0.f;
  if (blocks > 1) cluster_sync();   // nobody ends while another block may read its counts
}

// The rows to other pages, in the order of their places: blockIdx.x is the head, blockIdx.y the first of its runs of places
// (one list of all heads' rows, with a division for each: 66 us for 64 sequences of 8 heads cut to 2048 keys, 61 so).
template <int D, bool Q4>
__global__ void __launch_bounds__(256) evict_move_kernel(const __grid_constant__ EvictArgs a) {
  using R = RowParts<D, Q4>;
  constexpr int PER = 256 / R::LANES, AHEAD = 4;
  const R part(a.c, threadIdx.x % R::LANES);
  const unsigned bh = blockIdx.x;
  const int b = bh / a.c.Hkv, h = bh % a.c.Hkv, mine = threadIdx.x / R::LANES;
  wait_for_kernel_before();
  const int32_t* kept = a.kept + (size_t)bh * a.keep;
  const int left = (int)a.new_lengths[b];
  for (int first = blockIdx.y * (PER * AHEAD) + mine; first < left; first += gridDim.y * (PER * AHEAD)) {
    int j[AHEAD];
#pragma unroll
    for (int k = 0; k < AHEAD; ++k) j[k] = first + k * PER < left ? kept[first + k * PER] : -1;
    typename R::Data x[AHEAD];
#pragma unroll
    for (int k = 0; k < AHEAD; ++k)
      if (j[k] >= 0) x[k] = part.load(place_of<true>(a, a.from, bh, b, h, j[k]));
#pragma unroll
    for (int k = 0; k < AHEAD; ++k) {
      const long long to = j[k] >= 0 ? place_of<true>(a, a.to, bh, b, h, first + k * PER) : -1;
      if (to >= 0) part.store(to, x[k]);
    }
  }
}

template <int D, bool Q4, bool PAGED, bool MOVE>
cudaError_t launch_evict(const EvictArgs& a, long long heads, int blocks, cudaStream_t st) {
  cudaLaunchAttribute at{};
  at.id = cudaLaunchAttributeClusterDimension;
  at.val.clusterDim.x = blocks;
  at.val.clusterDim.y = at.val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)(heads * blocks));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = (size_t)a.cached * 4;
  cfg.stream = st;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  auto kernel = evict_kernel<D, Q4, PAGED, MOVE>;
  static std::atomic<uint64_t> allowed{0};
  cudaError_t e = blocks > 8 ? allow(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1, allowed) : cudaSuccess;
  if (e != cudaSuccess) return e;
  e = cudaLaunchKernelEx(&cfg, kernel, a);
  count_launches(1);
  if constexpr (!MOVE) {
    if (e != cudaSuccess) return e;
    constexpr int PER = 256 / RowParts<D, Q4>::LANES * 4;
    const int runs = (a.keep + PER - 1) / PER;
    e = launch_after(evict_move_kernel<D, Q4>, dim3((unsigned)heads, runs < 65535 ? runs : 65535), 256, st, a);
    count_launches(1);
  }
  return e;
}

// Whether two tables of the same sequences have an entry of memory in common.
bool share_entries(const fa_pages& x, const fa_pages& y) {
  const long long sx = x.B > 1 ? x.stride : x.M, sy = y.B > 1 ? y.stride : y.M;
  const long long off = ((long long)(intptr_t)y.table - (long long)(intptr_t)x.table) / 4;   // both are 4-byte aligned
  if (off >= sx * (x.B - 1) + x.M || off + sy * (y.B - 1) + y.M <= 0) return false;
  for (int b = 0; b < y.B; ++b) {
    const long long from = off + b * sy, past = from + y.M;   // of y's row b, in entries from x's first on
    const long long row = from < 0 ? -1 : from / sx;          // x's last row that begins at or before it
    if (row >= 0 && row < x.B && from - row * sx < x.M) return true;
    if (row + 1 < x.B && (row + 1) * sx < past) return true;
  }
  return false;
}

}  // namespace
}  // namespace fa

using namespace fa;

extern "C" fa_status fa_cache_evict(const fa_evict_params* p, const fa_cache* c, const fa_pages* pages, const fa_pages* to,
                                    const float* weights, int64_t W, const int64_t* lengths, float* weights_out,
                                    int32_t* kept, int64_t* new_lengths, void* stream) {
  clear_error();
  if (p == nullptr) { set_error("params is NULL"); return FA_ERR_INVALID_ARG; }
  CacheView held, cv, there;
  PageView from, dst;
  Span in[4], out[7];
  fa_status st = check_paged(c, pages, held, cv, from, in[0]);
  if (st != FA_OK) return st;
  if (to != nullptr && pages == nullptr) { set_error("a second table needs a first one"); return FA_ERR_INVALID_ARG; }
  if ((st = check_paged(c, to != nullptr ? to : pages, held, there, dst, in[1])) != FA_OK) return st;
  if (there.B != cv.B) { set_error("tables of %d and %d sequences", cv.B, there.B); return FA_ERR_INVALID_ARG; }
  if (p->reserved != 0) { set_error("reserved field must be 0"); return FA_ERR_INVALID_ARG; }
  if (p->keep < 1 || p->keep > kMaxSeq) { set_error("keep=%d outside [1, %d]", p->keep, kMaxSeq); return FA_ERR_INVALID_ARG; }
  if (p->sinks < 0 || p->recent < 0 || (long long)p->sinks + p->recent > p->keep) {
    set_error("sinks=%d, recent=%d: not negative, together at most keep=%d", p->sinks, p->recent, p->keep); return FA_ERR_INVALID_ARG;
  }
  if (to != nullptr && there.S < p->keep) {
    set_error("the second table has room for %d keys of %d", there.S, p->keep); return FA_ERR_INVALID_ARG;
  }
  // the same table again: in place
  const bool move = to == nullptr || (to->table == pages->table && (to->B == 1 || to->stride == pages->stride));
  if (!move && share_entries(*pages, *to)) { set_error("the two tables share entries"); return FA_ERR_INVALID_ARG; }
  if (W < 1 || W > 1LL << 30) { set_error("W=%lld outside [1, 2^30]", (long long)W); return FA_ERR_INVALID_ARG; }
  const long long heads = (long long)cv.B * cv.Hkv;
  if (heads * p->keep > 0x7fffffffLL - 512) { set_error("too many heads for one launch"); return FA_ERR_UNSUPPORTED; }
  const size_t bytes = (size_t)heads * (size_t)W * 4;
  in[2] = {lengths, (size_t)cv.B * 8, "lengths"};
  in[3] = {weights, weights != weights_out ? bytes : 0, "weights"};
  cache_spans(held, out);
  out[4] = {weights_out, bytes, "weights_out"};
  out[5] = {kept, (size_t)heads * p->keep * 4, "kept"};
  out[6] = {new_lengths, (size_t)cv.B * 8, "new_lengths"};
  if (lengths == nullptr || new_lengths == nullptr || (uintptr_t)lengths % 8 != 0 || (uintptr_t)new_lengths % 8 != 0) {
    set_error("lengths and new_lengths: there, and 8-byte aligned"); return FA_ERR_INVALID_ARG;
  }
  if (weights == nullptr || (uintptr_t)weights % 16 != 0) { set_error("weights is NULL or not 16-byte aligned"); return FA_ERR_INVALID_ARG; }
  if ((st = check_buffers(nullptr, 0, out, 6)) != FA_OK) return st;
  if ((st = check_apart(out, 6, out + 6, 1)) != FA_OK) return st;
  if ((st = check_apart(in, 4, out, 7)) != FA_OK) return st;
  EvictArgs a{};
  a.c = cv;
  a.from = from;
  a.to = dst;
  a.weights = weights;
  a.lengths = lengths;
  a.weights_out = weights_out;
  a.kept = kept;
  a.new_lengths = new_lengths;
  a.status = device_status_ptr();
  a.W = W;
  a.keep = p->keep;
  a.sinks = p->sinks;
  a.recent = p->recent;
  // As many blocks for a head as fill the SMs, none with less than 1024 keys.
  const long long keys = W < cv.S ? W : cv.S;
  int blocks = 1;
  while (blocks < kCluster && heads * blocks * 2 <= 2LL * sm_count() && keys >= 2048LL * blocks) blocks *= 2;
  const long long per = (keys + blocks - 1) / blocks;
  a.cached = (int)(per < kCached ? per : kCached);
  auto go = [&](auto dim, auto q4) {
    constexpr int D = decltype(dim)::value;
    constexpr bool Q4 = decltype(q4)::value;
    cudaStream_t cs = (cudaStream_t)stream;
    if (!move) return launch_evict<D, Q4, true, false>(a, heads, blocks, cs);
    return pages != nullptr ? launch_evict<D, Q4, true, true>(a, heads, blocks, cs) : launch_evict<D, Q4, false, true>(a, heads, blocks, cs);
  };
  using D64 = std::integral_constant<int, 64>;
  using D128 = std::integral_constant<int, 128>;
  cudaError_t e;
  if (cv.q4) e = cv.D == 64 ? go(D64{}, std::true_type{}) : go(D128{}, std::true_type{});
  else e = cv.D == 64 ? go(D64{}, std::false_type{}) : go(D128{}, std::false_type{});
  return cuda_status(e, "cache evict launch");
}
