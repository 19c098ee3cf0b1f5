// The attention weight that every key of a quantized cache got from a chunk of new tokens (fa_cache_weights).
//
// Mathematics. P_ij = exp(scale <q_i, k_j> - lse_i) summed over the rows i (tokens and query heads of the key's head) that see
// key j. With K as the left operand the products S^T = K Q^T have a key for each lane of TMEM and a row for each column, so
// that a thread adds up a key's weights along its lane, in registers: no atomics, no second pass, a fixed order.
//
// A block has one tile of 128 keys of a sequence's head: warps 0-7 make its bf16 operand from the packed bytes (kv_tile.cuh);
// then warps 0-3 own a key for each thread, warps 4-7 bring the rows, 128 (or 16, where there are no more) at a time, and one
// thread of warp 8 issues the MMAs; the products are in two buffers, so that they and the exponentials overlap.
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
constexpr int kThreads = 288;

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
  float sl2;         // |scale| log2(e); the sign, or a scale of 0, is in the two masks
  uint32_t q_and, q_xor;
  int Hq, Sq, window, layout, G;
};

template <int D, int NQ>
struct WeightSmem {
  static constexpr int kBox = 128 * 128;               // 64 features of 128 rows
  static constexpr int kK = 128 * D * 2;
  static constexpr int kQBox = NQ * 128, kQ = NQ * D * 2;
  static constexpr int kQOff = kK, kLogOff = kQOff + 2 * kQ, kPosOff = kLogOff + 2 * NQ * 4, kBarOff = kPosOff + 2 * NQ * 4;
  static constexpr int kBytes = kBarOff + 128 + 1024;
  static constexpr int kColumns = NQ < 32 ? 64 : 2 * NQ;   // of TMEM
};

template <int D, bool Q4, bool PAGED, int NQ>
__global__ void __launch_bounds__(kThreads) weights_kernel(const __grid_constant__ WeightArgs a) {
  using L = WeightSmem<D, NQ>;
  constexpr int STEP = L::kColumns / 2;   // columns from one buffer of products to the other
  extern __shared__ uint8_t smem_raw[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int heads = a.c.B * a.c.Hkv;
  const int bh = blockIdx.x % heads, b = bh / a.c.Hkv, h = bh % a.c.Hkv;
  const int key0 = blockIdx.x / heads * kTileKeys;

  const long long length = a.lengths != nullptr ? __ldg(a.lengths + b) : a.c.S;
  const long long tokens = a.count != nullptr ? __ldg(a.count + b) : a.Sq;
  const int len = (int)min(max(length, 0LL), (long long)a.c.S), n = (int)min(max(tokens, 0LL), (long long)a.Sq);
  if (key0 == 0 && h == 0 && threadIdx.x == 0 && (len != length || n != tokens || len > a.W) && a.status != nullptr)
    atomicCAS(a.status, 0u, 0x40000000u | kSiteDecodeLength);
  // the rows that see one of the keys: tokens [first, last]
  const int before = len - n;
  const int first = max(key0 - before, 0);
  const int last = a.window > 0 ? min(n - 1, min(key0 + kTileKeys, len) - 1 + a.window - before) : n - 1;
  const int row0 = first * a.G, rows = key0 < len ? max((last + 1) * a.G - row0, 0) : 0;
  float sum = 0.f;

  if (rows > 0) {   // the whole block has one answer
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const uint32_t sK = smem_u32(smem), sQ = smem_u32(smem + L::kQOff);
    float* sLog = reinterpret_cast<float*>(smem + L::kLogOff);   // [2][NQ]: -lse, base 2; -inf in columns without a row
    int* sPos = reinterpret_cast<int*>(smem + L::kPosOff);       // [2][NQ]
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + L::kBarOff);
    uint64_t* bar_k = bars;          // K written
    uint64_t* bar_q = bars + 1;      // [2]: rows written
    uint64_t* bar_s = bars + 3;      // [2]: products there
    uint64_t* bar_free = bars + 5;   // [2]: products and rows read
    uint64_t* bar_done = bars + 7;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 8);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
    if (threadIdx.x == 0) {
      mbar_init(bar_k, 8);
      for (int i = 0; i < 2; ++i) {
        mbar_init(&bar_q[i], 4);
        mbar_init(&bar_s[i], 1);
        mbar_init(&bar_free[i], 4);
      }
      mbar_init(bar_done, 1);
      *abort_flag = 0;
      fence_barrier_init();
    }
    if (warp == 8) tmem_alloc(tmem_slot, L::kColumns);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    const int tiles = (rows + NQ - 1) / NQ;

    if (warp < 8) {   // this warp's run of K
      const int run = key0 + kRun * warp;
      long long row = -1;
      if (run < len) row = PAGED ? page_row(a.pages, a.c.Hkv, b, h, run, a.status) : (long long)bh * a.c.S + run;
      RunBytes<D, Q4> k;
      k.load(a.c.k_q, a.c.k_d, row, min(len - run, kRun));
      k.store(sK, warp, false);
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar_k);
    }
    if (warp < 4) {
      const int key = key0 + 32 * warp + lane;
      const uint32_t tS = tmem + ((uint32_t)(warp * 32) << 16);
      const uint64_t sl2 = f32x2(a.sl2, a.sl2);
      for (int i = 0; i < tiles; ++i) {
        const int buf = i & 1;
        if (!__all_sync(0xffffffffu, mbar_wait<true>(&bar_s[buf], (i >> 1) & 1, abort_flag, a.status, 1101))) break;
        tc_fence_after();
        const float* log = sLog + buf * NQ;
        const int* pos = sPos + buf * NQ;
        const int here = min(rows - i * NQ, NQ);
        const bool edge = pos[0] < key0 + kTileKeys - 1 || (a.window > 0 && pos[here - 1] - key0 > a.window);
        uint64_t part[2] = {f32x2(0.f, 0.f), f32x2(0.f, 0.f)};
        auto add = [&](const auto& raw, int c0, auto on_edge) {
          constexpr int N = sizeof(raw) / 4;
#pragma unroll
          for (int e = 0; e < N; e += 4) {
            const float4 g = *reinterpret_cast<const float4*>(log + c0 + e);
            const float gs[4] = {g.x, g.y, g.z, g.w};
#pragma unroll
            for (int k = 0; k < 4; k += 2) {
              float t0, t1;
              f32x2_split(fma_f32x2(f32x2(__uint_as_float(raw[e + k]), __uint_as_float(raw[e + k + 1])), sl2, f32x2(gs[k], gs[k + 1])), t0, t1);
              float p0 = ex2_approx(t0), p1 = ex2_approx(t1);
              if constexpr (decltype(on_edge)::value) {
                const int at0 = pos[c0 + e + k], at1 = pos[c0 + e + k + 1];
                if (key > at0 || (a.window > 0 && at0 - key > a.window)) p0 = 0.f;
                if (key > at1 || (a.window > 0 && at1 - key > a.window)) p1 = 0.f;
              }
              part[k / 2] = add_f32x2(part[k / 2], f32x2(p0, p1));
            }
          }
        };
        auto all = [&](auto on_edge) {
          if constexpr (NQ == 16) {
            uint32_t raw[16];
            tmem_ld16(tS + buf * STEP, raw);
            tmem_wait_ld();
            reg_fence16(raw);
            add(raw, 0, on_edge);
          } else {
#pragma unroll 1
            for (int c0 = 0; c0 < here; c0 += 32) {
              uint32_t raw[32];
              tmem_ld32(tS + buf * STEP + c0, raw);
              tmem_wait_ld();
              reg_fence(raw);
              add(raw, c0, on_edge);
            }
          }
        };
        if (edge) all(std::true_type{});
        else all(std::false_type{});
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bar_free[buf]);
        float s0, s1, s2, s3;
        f32x2_split(part[0], s0, s1);
        f32x2_split(part[1], s2, s3);
        sum += (s0 + s1) + (s2 + s3);
      }
    } else if (warp < 8) {
      const int r = threadIdx.x - 128;   // the row of a tile that this thread brings
      for (int i = 0; i < tiles; ++i) {
        const int buf = i & 1;
        if (i >= 2 && !__all_sync(0xffffffffu, mbar_wait<true>(&bar_free[buf], ((i >> 1) - 1) & 1, abort_flag, a.status, 1102))) break;
        if (r < NQ) {
          const int row = row0 + i * NQ + r, token = row / a.G;
          const bool on = i * NQ + r < rows;
          const int head = h * a.G + row % a.G;
          const size_t at = on ? (a.layout ? ((size_t)b * a.Sq + token) * a.Hq + head : ((size_t)b * a.Hq + head) * a.Sq + token) * D : 0;
          const uint4* src = reinterpret_cast<const uint4*>(a.q + at);
          const uint32_t dst = sQ + buf * L::kQ + r * 128;
          const float log = on ? __ldg(a.lse + ((size_t)b * a.Hq + head) * a.Sq + token) : 0.f;
#pragma unroll
          for (int c0 = 0; c0 < D / 8; c0 += 8) {
            uint4 u[8];
#pragma unroll
            for (int c = 0; c < 8; ++c) u[c] = on ? __ldg(src + c0 + c) : make_uint4(0, 0, 0, 0);
#pragma unroll
            for (int c = 0; c < 8; ++c)
              st_shared_v4(dst + (c0 / 8) * L::kQBox + ((c ^ (r & 7)) << 4), (u[c].x & a.q_and) ^ a.q_xor,
                           (u[c].y & a.q_and) ^ a.q_xor, (u[c].z & a.q_and) ^ a.q_xor, (u[c].w & a.q_and) ^ a.q_xor);
          }
          sLog[buf * NQ + r] = on ? -log * kLog2e : -CUDART_INF_F;
          sPos[buf * NQ + r] = on ? before + token : -1;
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bar_q[buf]);
      }
    } else if (lane == 0) {
      const uint32_t idesc = idesc_bf16_f32(128, NQ, 0, 0);
      bool ok = mbar_wait<true>(bar_k, 0, abort_flag, a.status, 1103);
      const uint64_t dk0 = smem_desc_sw128(sK, 16, 1024);
      for (int i = 0; ok && i < tiles; ++i) {
        const int buf = i & 1;
        if (!(ok = mbar_wait<true>(&bar_q[buf], (i >> 1) & 1, abort_flag, a.status, 1104))) break;
        tc_fence_after();
        const uint64_t dq0 = smem_desc_sw128(sQ + buf * L::kQ, 16, 1024);
#pragma unroll
        for (int k = 0; k < D / 16; ++k)
          mma_ss(tmem + buf * STEP, desc_add(dk0, (k >> 2) * L::kBox + (k & 3) * 32),
                 desc_add(dq0, (k >> 2) * L::kQBox + (k & 3) * 32), idesc, k > 0 ? 1u : 0u);
        mma_commit(&bar_s[buf]);
      }
      mma_commit(bar_done);
      mbar_wait<true>(bar_done, 0, nullptr, a.status, 1105);
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    if (warp == 8) {
      tc_fence_after();
      tmem_dealloc(tmem, L::kColumns);
    }
  }
  const long long key = (long long)key0 + threadIdx.x;
  if (warp < 4 && key < a.W) {
    const size_t at = (size_t)bh * a.W + key;
    a.out[at] = (a.weights != nullptr ? a.weights[at] : 0.f) + sum;
  }
}

template <int D, bool Q4, bool PAGED, int NQ>
cudaError_t launch_weights(const WeightArgs& a, unsigned blocks, cudaStream_t st) {
  constexpr int bytes = WeightSmem<D, NQ>::kBytes;
  auto kernel = weights_kernel<D, Q4, PAGED, NQ>;
  static std::atomic<uint64_t> allowed{0};
  const cudaError_t e = allow_shared(kernel, bytes, allowed);
  if (e != cudaSuccess) return e;
  kernel<<<blocks, kThreads, bytes, st>>>(a);
  count_launches(1);
  return cudaGetLastError();
}

}  // namespace
}  // namespace fa

using namespace fa;

extern "C" fa_status fa_cache_weights(const fa_prefill_params* p, const void* q, const float* lse, const fa_cache* c,
                                      const fa_pages* pages, const int64_t* lengths, const int64_t* count,
                                      const float* weights, int64_t W, float* out, void* stream) {
  clear_error();
  if (p == nullptr) { set_error("params is NULL"); return FA_ERR_INVALID_ARG; }
  CacheView held, cv;
  PageView pv;
  Span in[8], planes[4], outs[1];
  fa_status st = check_paged(c, pages, held, cv, pv, in[4]);
  if (st != FA_OK) return st;
  if ((st = check_chunk(p, cv)) != FA_OK) return st;
  const long long heads = (long long)cv.B * cv.Hkv;
  if (W < 1 || W > (1LL << 31) - kTileKeys) { set_error("W=%lld outside [1, 2^31 - 128]", (long long)W); return FA_ERR_INVALID_ARG; }
  const long long blocks = (W + kTileKeys - 1) / kTileKeys * heads;
  if (blocks > 0x7fffffffLL) { set_error("too many keys for one launch"); return FA_ERR_UNSUPPORTED; }
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
  a.sl2 = p->scale == 0.f ? 1.f : fminf(fabsf(p->scale) * kLog2e, FLT_MAX);
  a.q_and = p->scale == 0.f ? 0u : 0xffffffffu;
  a.q_xor = p->scale < 0.f ? 0x80008000u : 0u;
  a.Hq = p->Hq;
  a.Sq = p->Sq;
  a.window = p->window < 2 * kMaxSeq ? p->window : 2 * kMaxSeq;
  a.layout = p->layout;
  a.G = p->Hq / cv.Hkv;
  const bool few = (long long)a.G * p->Sq <= 16;
  auto go = [&](auto dim, auto q4) {
    constexpr int D = decltype(dim)::value;
    constexpr bool Q4 = decltype(q4)::value;
    const unsigned n = (unsigned)blocks;
    cudaStream_t cs = (cudaStream_t)stream;
    if (pages != nullptr) return few ? launch_weights<D, Q4, true, 16>(a, n, cs) : launch_weights<D, Q4, true, 128>(a, n, cs);
    return few ? launch_weights<D, Q4, false, 16>(a, n, cs) : launch_weights<D, Q4, false, 128>(a, n, cs);
  };
  using D64 = std::integral_constant<int, 64>;
  using D128 = std::integral_constant<int, 128>;
  cudaError_t e;
  if (cv.q4) e = cv.D == 64 ? go(D64{}, std::true_type{}) : go(D128{}, std::true_type{});
  else e = cv.D == 64 ? go(D64{}, std::false_type{}) : go(D128{}, std::false_type{});
  return cuda_status(e, "cache weights launch");
}
