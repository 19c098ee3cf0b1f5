// Attention of a chunk of new tokens of every sequence, a ragged batch, over its quantized cache, in pages or in one piece
// (fa_prefill): the serving form of the forward, on the 5th-generation tensor cores.
//
// Mathematics. The G = Hq / Hkv query heads of a key/value head and its tokens are the rows of one matrix, token by token, so
// that a tile of 128 rows covers few positions and skips what lies behind the last. With K and V rounded to bf16:
// S = scale Q K^T, hidden pairs -inf, O = softmax(S) V by tiles of 128 keys with a running reference and sum, in 32 bits; P is
// rounded to bf16 for its product, which has fp32's range: so the reference is any number near the maximum, is set by a unit's
// first 32 scores, and follows only when the maximum is more than 2^30 above it. Weights, sums and O hold that without loss (O
// stays below 2^30 * 2^24 keys * 2^23), and scores are read once, with nothing to wait for between their maximum and their exponentials.
//
// Split. A unit is 256 rows (two tiles) of one sequence's key/value head. The tiles of 128 keys of all units form one list,
// cut into equal slices, one for each SM: the end of one unit, whole units, the beginning of another. A unit that several
// slices share leaves its parts (unnormalised O, reference and sum) in the workspace, and a second kernel joins them. So one
// row block over a long window and a batch of short ones fill the machine alike, without a choice of splits; a block
// finds its place in the list from the lengths, on the device.
//
// A block of 20 warps. Warp 0 issues the MMAs (S_t = Q_t K^T, O_t += P_t V) and walks the list for all. Eight warps read the
// packed bytes and write the bf16 operands (kv_tile.cuh), a run of 16 keys each, one tile of K and the V of the tile before into
// each stage of a ring. Warps 1-3 bring Q_0 and
// Q_1, as soon as the last product with the ones before is done. Warps 12-15 and 16-19 have a row of Q_0 and Q_1 for each thread:
// they turn scores into P in TMEM, and write O at the end. They hold 32 scores at a time: a row of
// 128 in registers leaves so few to the others that these spill, and what is spilled is in L2, as shared memory takes what L1 has.
// TMEM (512 columns): S0 [0,128), S1 [128,256), O0 [256, 256+D), O1 [256+D, 256+2D).
//
// Measured (device time, captured calls over changing inputs): 512 tokens over 67,584 keys in 4 bits, 16 heads on 4, D = 128: 253 us,
// 1.12 PFLOP/s, 58% of the measured dense rate; two prompts of 4096 tokens in 8 bits, 32 heads on 8: 337 to 343 us, 0.8 PFLOP/s of visible
// pairs; 24 tokens of 8 sequences of 500 to 4000 keys in 4 bits: 33 us; chunks of 1 to 777 tokens of 6 sequences of 300 to 9000 keys in 8
// bits, D = 64, in a sliding window of 1024: 51 us. What bounds it: a tile of keys and 256 rows takes 4400 cycles, of which the
// tensor cores are busy for half: each tile of rows goes from S to softmax (2400 cycles for 128 scores a row) to P V and back, and two of them on that way
// do not fill the pipe; in copies without softmax the first case takes 204 us, without operands made from bytes as well 169. With few
// tokens it is the way: 2.7 us for the list, 1.5 to the first bytes, 1.5 to 2 for each tile of keys, 1.5 for O, and the join.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cfloat>
#include <cmath>
#include <type_traits>

#include "fa_check.h"
#include "fa_device.cuh"
#include "kv_tile.cuh"
#include "tc_ptx.cuh"

namespace fa {
namespace {

using namespace tc;

constexpr int kBM = 128;          // rows of a tile
constexpr int kUnit = 2 * kBM;    // rows of a unit
constexpr int kBN = kTileKeys;
constexpr int kThreads = 640;
constexpr int kLoaders = 8;       // warps that make operands
constexpr int kListed = 1024;     // sequences of a launch; more are more launches
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kRescale = 30.f;   // log2 units: the reference follows the maximum when that is more above it
// Registers of a thread: what 640 are launched with, and what warps 0-11 and those that have rows make of it.
constexpr int kRegsLaunch = 96, kRegsLoad = 80, kRegsSoftmax = 120;
static_assert(3 * kRegsLoad + 2 * kRegsSoftmax <= 5 * kRegsLaunch, "register split exceeds the launch's");

struct Record {   // a unit that slices c0 .. c1 share (c1 < 0: none)
  int b, h, unit, rows, c0, c1, padding[2];
};

struct PrefillArgs {
  CacheView c;
  PageView pages;
  const __nv_bfloat16* q;
  __nv_bfloat16* o;
  float* lse;
  const int64_t* lengths;
  const int64_t* count;
  float* part_o;     // [slices, 2, part_rows, D], unnormalised: of the unit a slice begins inside of, of the one it ends in
  float2* part_ml;   // [slices, 2, part_rows]: what the weights are relative to (base 2), and their sum
  Record* records;   // [slices]: the unit that a slice is the second of
  unsigned* status;
  float sl2;         // |scale| log2(e); the sign, or a scale of 0, is in the two masks
  uint32_t q_and, q_xor;
  int Hq, Sq, window, layout, G, part_rows;
  bool wide;         // o is 32-byte aligned
};

// A sequence's keys and tokens.
struct Seq { int len, n; };

__device__ __forceinline__ Seq seq_of(const PrefillArgs& a, int b, bool report) {
  const long long len = a.lengths != nullptr ? __ldg(a.lengths + b) : a.c.S;
  const long long n = a.count != nullptr ? __ldg(a.count + b) : a.Sq;
  const Seq s{(int)min(max(len, 0LL), (long long)a.c.S), (int)min(max(n, 0LL), (long long)a.Sq)};
  if (report && (s.len != len || s.n != n) && a.status != nullptr) atomicCAS(a.status, 0u, 0x40000000u | kSiteDecodeLength);
  return s;
}

__device__ __forceinline__ int units_of(const PrefillArgs& a, Seq s) { return (s.n * a.G + kUnit - 1) / kUnit; }

// The tiles of keys that a unit's rows see: at least one, so that rows which see nothing are written by someone.
struct Tiles { int begin, end; };

__device__ __forceinline__ Tiles tiles_of(const PrefillArgs& a, Seq s, int unit) {
  const int first = unit * kUnit / a.G, last = (min(unit * kUnit + kUnit, s.n * a.G) - 1) / a.G;   // tokens
  const int before = s.len - s.n;
  Tiles t;
  t.begin = a.window > 0 ? max(before + first - a.window, 0) / kBN : 0;
  t.end = max((max(before + last + 1, 0) + kBN - 1) / kBN, t.begin + 1);
  return t;
}

// `total` tiles cut into n slices that differ by one at most, the larger ones first.
struct Slices {
  long long each, more;
  __device__ __forceinline__ Slices(long long total, int n) : each(total / n), more(total % n) {}
  __device__ __forceinline__ long long begin(long long i) const { return i * each + min(i, more); }
  __device__ __forceinline__ int of(long long tile) const {
    const long long large = more * (each + 1);
    return (int)(tile < large ? tile / (each + 1) : more + (tile - large) / each);
  }
};

// What every role of a block knows of the list.
struct Plan {
  Seq seq[kListed];
  long long before[kListed + 1];   // tiles of the sequences before, all heads
  int b, h, unit, off;             // where the slice begins
  long long tiles;                 // how many it has
};

__device__ __forceinline__ long long warp_sum_ll(long long x) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}

// Fills the plan (all threads of the block).
__device__ __forceinline__ void make_plan(const PrefillArgs& a, Plan& plan, int slice, int slices) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  for (int b = threadIdx.x; b < a.c.B; b += kThreads) plan.seq[b] = seq_of(a, b, slice == 0);
  __syncthreads();
  for (int b = warp; b < a.c.B; b += kThreads / 32) {
    const Seq s = plan.seq[b];
    const int n = units_of(a, s);
    long long x = 0;
    for (int u = lane; u < n; u += 32) {
      const Tiles t = tiles_of(a, s, u);
      x += t.end - t.begin;
    }
    x = warp_sum_ll(x);
    if (lane == 0) plan.before[b] = x * a.c.Hkv;
  }
  __syncthreads();
  if (warp != 0) {
    __syncthreads();
    return;
  }
  long long all = 0;   // an exclusive sum in place
  for (int b0 = 0; b0 < a.c.B; b0 += 32) {
    const long long own = b0 + lane < a.c.B ? plan.before[b0 + lane] : 0;
    long long x = own;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    if (b0 + lane < a.c.B) plan.before[b0 + lane] = all + x - own;
    all += __shfl_sync(0xffffffffu, x, 31);
  }
  if (lane == 0) plan.before[a.c.B] = all;
  __syncwarp();
  const Slices cut(all, slices);
  const long long at = cut.begin(slice), tiles = cut.begin(slice + 1) - at;
  Record rec{0, 0, 0, 0, 0, -1, {0, 0}};
  if (tiles > 0) {
    int b = 0;   // the last sequence that begins at or before the slice; one without tiles begins where the next does
    for (int b0 = 0; b0 < a.c.B; b0 += 32) b += __popc(__ballot_sync(0xffffffffu, b0 + lane < a.c.B && plan.before[b0 + lane] <= at));
    --b;
    const Seq s = plan.seq[b];
    const long long head = (plan.before[b + 1] - plan.before[b]) / a.c.Hkv, off = at - plan.before[b];
    const int h = (int)(off / head), n = units_of(a, s);
    long long rest = off % head;   // tiles of the head before the slice
    int unit = 0, inside = 0, length = 0;
    for (int u0 = 0; u0 < n; u0 += 32) {
      const int u = u0 + lane;
      int own = 0;
      if (u < n) {
        const Tiles t = tiles_of(a, s, u);
        own = t.end - t.begin;
      }
      long long x = own;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const long long y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
      }
      const uint32_t past = __ballot_sync(0xffffffffu, x > rest);   // units that end behind the slice's first tile
      if (past != 0) {
        const int l = __ffs(past) - 1;
        unit = u0 + l;
        inside = (int)(rest - __shfl_sync(0xffffffffu, x - own, l));
        length = __shfl_sync(0xffffffffu, own, l);
        break;
      }
      rest -= __shfl_sync(0xffffffffu, x, 31);
    }
    if (lane == 0) {
      plan.b = b;
      plan.h = h;
      plan.unit = unit;
      plan.off = inside;
    }
    if (inside > 0 && cut.begin(slice - 1) <= at - inside)
      rec = Record{b, h, unit, min(s.n * a.G - unit * kUnit, kUnit), slice - 1, cut.of(at - inside + length - 1), {0, 0}};
  }
  if (lane == 0) {
    plan.tiles = tiles;
    if (a.records != nullptr) a.records[slice] = rec;
  }
  __syncthreads();
}

// A slice's part of one unit, as the roles of a block find it in shared memory: the issuing thread walks the list and writes
// the parts one after the other into a ring, four ahead, so that nobody else has the walk's state in registers.
struct Piece {
  int b, h, unit;
  int tile, tiles;      // the first one, and how many; none: the list has ended
  int rows;             // live rows of the unit
  int len, n;           // the sequence's keys and tokens
  int starts, ends;     // the unit's first, last tile is among them
};
constexpr int kPieces = 8;

struct Walk {
  const PrefillArgs& a;
  const Plan& plan;
  int b, h, unit, off;
  long long left;
  __device__ __forceinline__ Walk(const PrefillArgs& a_, const Plan& p)
      : a(a_), plan(p), b(p.b), h(p.h), unit(p.unit), off(p.off), left(p.tiles) {}
  __device__ __forceinline__ void next(Piece& x) {
    x.tiles = 0;
    if (left <= 0) return;
    const Seq s = plan.seq[b];
    const Tiles t = tiles_of(a, s, unit);
    x.b = b;
    x.h = h;
    x.unit = unit;
    x.tile = t.begin + off;
    x.rows = min(s.n * a.G - unit * kUnit, kUnit);
    x.len = s.len;
    x.n = s.n;
    const int tiles = (int)min((long long)(t.end - t.begin - off), left);
    x.starts = off == 0;
    x.ends = off + tiles == t.end - t.begin;
    x.tiles = tiles;
    left -= tiles;
    off = 0;
    if (++unit == units_of(a, s)) {
      unit = 0;
      if (++h == a.c.Hkv) {
        h = 0;
        do ++b;
        while (b < a.c.B && plan.seq[b].n == 0);
      }
    }
  }
};

// Element offset of a unit's row in q and o, and its place in lse.
struct RowPlace {
  int token;
  size_t at, log;
};
__device__ __forceinline__ RowPlace place_of(const PrefillArgs& a, int b, int h, int row) {
  const int i = row / a.G, head = h * a.G + row % a.G;
  RowPlace p;
  p.token = i;
  p.at = (a.layout ? ((size_t)b * a.Sq + i) * a.Hq + head : ((size_t)b * a.Hq + head) * a.Sq + i) * a.c.D;
  p.log = ((size_t)b * a.Hq + head) * a.Sq + i;
  return p;
}

// 32 bytes: a sector of L2 whole where they are one (two prompts of 4096 tokens in 8 bits: 371 us in halves, 349 so).
__device__ __forceinline__ void st_global_32(bool whole, uint4* p, uint32_t a, uint32_t b, uint32_t c, uint32_t d, uint32_t e, uint32_t f,
                                             uint32_t g, uint32_t h) {
  if (!whole) {
    p[0] = make_uint4(a, b, c, d);
    p[1] = make_uint4(e, f, g, h);
    return;
  }
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(a), "r"(b), "r"(c), "r"(d), "r"(e), "r"(f),
               "r"(g), "r"(h) : "memory");
}

template <int D>
struct PrefillSmem {
  static constexpr int kBoxBytes = 128 * 128;
  static constexpr int kTileBytes = kBM * D * 2;
  static constexpr int kStages = D == 128 ? 2 : 4;   // a stage: the V of one tile of keys and the K of the next
  static constexpr int kKVOff = 2 * kTileBytes;
  static constexpr int kBarOff = kKVOff + 2 * kStages * kTileBytes;
  static constexpr int kPieceOff = kBarOff + 320;
  static constexpr int kPlanOff = kPieceOff + 384;
  static constexpr int kBytes = kPlanOff + (int)sizeof(Plan) + 1024;
};

// ALONE: no unit has more than one tile of rows. Such a tile has both buffers of S: its next scores are made, and softmax goes on to
// them, while its product is (24 tokens of 8 sequences: 32.8 us, 35.5 without; of one of 67,584 keys, 4 heads: 43.1 and 49.8).
template <int D, bool Q4, bool PAGED, bool ALONE>
__global__ void __launch_bounds__(kThreads, 1) prefill_kernel(const __grid_constant__ PrefillArgs a) {
  using L = PrefillSmem<D>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sQ = smem_u32(smem), sKV = smem_u32(smem + L::kKVOff);
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + L::kBarOff);
  uint64_t* bar_q = bars;                         // [2]: tile t of a unit's Q written
  uint64_t* bar_s = bars + 2;                     // [2]: scores of tile t there; ALONE: of even and odd tiles of keys
  uint64_t* bar_p = bars + 4;                     // [2]: weights there, likewise
  uint64_t* bar_o = bars + 6;                     // [2]: the last product of tile t done
  uint64_t* bar_v = bars + 8;                     // [2], ALONE: an even, an odd product done
  uint64_t* bar_full = bars + 10;                 // [kStages]: stage written
  uint64_t* bar_empty = bar_full + L::kStages;    // [kStages]: its MMAs done
  uint64_t* bar_piece = bar_empty + L::kStages;   // [kPieces]: part of a unit described
  uint64_t* bar_past = bar_piece + kPieces;       // [kPieces]: nobody looks at it any more
  uint64_t* bar_read = bar_past + kPieces;        // [2]: the last product with tile t of a unit's Q done
  uint64_t* bar_done = bar_read + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bar_done + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  static_assert(8 * (10 + 2 * L::kStages + 2 * kPieces + 3) + 8 <= 256 + 64 && kPieces * sizeof(Piece) <= 320, "shared memory of barriers and parts");
  Piece* pieces = reinterpret_cast<Piece*>(smem + L::kPieceOff);
  Plan& plan = *reinterpret_cast<Plan*>(smem + L::kPlanOff);
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;

  let_next_kernel_start();
  if (threadIdx.x == 0) {
    for (int t = 0; t < 2; ++t) {
      mbar_init(&bar_q[t], 3);
      mbar_init(&bar_read[t], 1);
      mbar_init(&bar_s[t], 1);
      mbar_init(&bar_p[t], 4);
      mbar_init(&bar_o[t], 1);
      mbar_init(&bar_v[t], 1);
    }
    for (int i = 0; i < L::kStages; ++i) {
      mbar_init(&bar_full[i], kLoaders);
      mbar_init(&bar_empty[i], 1);
    }
    for (int i = 0; i < kPieces; ++i) {
      mbar_init(&bar_piece[i], 1);
      mbar_init(&bar_past[i], 3 + kLoaders + 8);   // the warps that bring Q, that load and that have rows
    }
    mbar_init(bar_done, 1);
    *abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == 0) tmem_alloc(tmem_slot, 512);
  make_plan(a, plan, blockIdx.x, gridDim.x);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, *tmem_slot, 0);   // one number to the compiler too
  // part i of the slice is there (all lanes of a warp have one answer)
  auto part_there = [&](int i) { return mbar_wait<true>(&bar_piece[i % kPieces], (i / kPieces) & 1, abort_flag, a.status, 1009); };

  if (warp < 12) {
    regs_dec<kRegsLoad>();
    if (warp == 0) {
      // ---------------------------------------------------------------- the list, and the MMAs
      // All lanes go this way together, and the first issues: descriptors then are the warp's, in uniform registers, where
      // the issue of one lane alone takes each word there first (and is what the tensor cores wait for).
      const uint32_t lead = lane == 0 ? 1u : 0u;
      Walk walk(a, plan);
      int listed = 0;
      bool listed_all = false, ok = true;
      auto list_part = [&] {   // one more
        if (listed_all || !ok) return;
        if (listed >= kPieces &&
            !(ok = mbar_wait_warp(&bar_past[listed % kPieces], (listed / kPieces - 1) & 1, abort_flag, a.status, 1010)))
          return;
        Piece x;
        walk.next(x);
        if (lane == 0) {
          pieces[listed % kPieces] = x;
          mbar_arrive(&bar_piece[listed % kPieces]);
        }
        __syncwarp();
        listed_all = __shfl_sync(0xffffffffu, x.tiles, 0) == 0;
        ++listed;
      };
      // Some parts ahead: a warp that loads looks at the tile behind the one that it completes the stage of, which may be
      // another part's; it would wait for that part, and this warp for the stage.
      for (int i = 0; i < 4; ++i) list_part();
      const uint32_t idesc_qk = idesc_bf16_f32(kBM, kBN, 0, 0);
      const uint32_t idesc_pv = idesc_bf16_f32(kBM, D, 0, 1);
      const uint64_t dq = smem_desc_sw128(sQ, 16, 1024), dk = smem_desc_sw128(sKV, 16, 1024), dv = smem_desc_sw128(sKV, L::kBoxBytes, 1024);
      // buffer b of S and P
      auto issue_pv = [&](int t, int b, int slot, bool first) {
        const uint64_t v = desc_add(dv, slot * L::kTileBytes);
#pragma unroll
        for (int k = 0; k < kBN / 16; ++k)
          mma_ts_if(lead, tmem + 256 + t * D, tmem + b * 128 + k * 8, desc_add(v, k * 2048), idesc_pv,
                    (!first || k > 0) ? 1u : 0u);
      };
      auto issue_s = [&](int t, int b, int slot) {
        const uint64_t q = desc_add(dq, t * L::kTileBytes), k0 = desc_add(dk, slot * L::kTileBytes);
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
          const uint32_t off = (k >> 2) * L::kBoxBytes + (k & 3) * 32;
          mma_ss_if(lead, tmem + b * 128, desc_add(q, off), desc_add(k0, off), idesc_qk, k > 0 ? 1u : 0u);
        }
        mma_commit_if(lead, &bar_s[b]);
      };
      auto wait = [&](uint64_t* bar, int phase, unsigned site) {
        return mbar_wait_warp(bar, phase & 1, abort_flag, a.status, site);
      };
      // The parts' tiles are one stream: stage i holds the K of its tile i and the V of tile i - 1. Within a part a tile of
      // rows gets its P V of the last tile of keys and then its next S, one tile of rows after the other; where a part ends
      // both products come first. ALONE: the next S into the other buffer, and then the product.
      int stage = 0;                    // tiles of the stream so far
      int scores0 = 0, scores1 = 0;     // of bar_s and bar_p: completions so far
      int loads0 = 0, loads1 = 0;       // of bar_q
      int pending = 0;                  // tiles of rows of the last tile of keys whose product is to come
      bool pending_first = false, pending_last = false;   // it is its part's first, last
      int pending_b = 0, products = 0;   // ALONE: its buffer; products so far
      auto product = [&](int t, int slot) -> bool {
        const int b = ALONE ? pending_b : t;
        if (!wait(&bar_p[b], (b ? scores1 : scores0) - 1, 1001)) return false;
        tc_fence_after();
        issue_pv(t, b, slot, pending_first);
        if (ALONE) mma_commit_if(lead, &bar_v[products++ & 1]);
        if (pending_last) mma_commit_if(lead, &bar_o[t]);
        return true;
      };
      auto scores = [&](int t, int b, int slot, bool last) {
        issue_s(t, b, slot);
        if (last) mma_commit_if(lead, &bar_read[t]);
        if (b) ++scores1;
        else ++scores0;
      };
      for (int i = 0; ok; ++i) {
        const int rows = __shfl_sync(0xffffffffu, pieces[i % kPieces].rows, 0);   // listed by this warp
        const int tiles = __shfl_sync(0xffffffffu, pieces[i % kPieces].tiles, 0);
        if (tiles == 0 && pending == 0) break;
        const int live = tiles == 0 ? 0 : rows > kBM ? 2 : 1;
        for (int j = 0; ok && j < max(tiles, 1); ++j) {   // behind the last part a stage that holds only V
          const int sb = stage % L::kStages;
          if (!(ok = wait(&bar_full[sb], stage / L::kStages, 1002))) break;
          // The last product but one has ended and is seen before more scores are made, so that who waits for the last one's barrier
          // meets it one completion short or complete, never two short, which a phase's parity cannot tell from complete.
          if (ALONE && products >= 2 && !(ok = wait(&bar_v[products & 1], products / 2 - 1, 1013))) break;
          tc_fence_after();
          const bool last = j == tiles - 1;
          if (j == 0) {   // rolled: what warps go through has to come from the instruction caches
#pragma unroll 1
            for (int x = 0; ok && x < 4; ++x) {
              const int t = x & 1;
              if (x < 2) {
                if (t < pending) ok = product(t, 2 * sb + 1);
              } else if (t < live) {
                if (!(ok = wait(&bar_q[t], t ? loads1 : loads0, 1003))) break;
                tc_fence_after();
                if (t) ++loads1;
                else ++loads0;
                scores(t, t, 2 * sb, last);
              }
            }
            list_part();
          } else if constexpr (ALONE) {
            scores(0, j & 1, 2 * sb, last);
            ok = product(0, 2 * sb + 1);
          } else {
            if ((ok = product(0, 2 * sb + 1))) scores(0, 0, 2 * sb, last);
            if (ok && live > 1 && (ok = product(1, 2 * sb + 1))) scores(1, 1, 2 * sb, last);
          }
          if (!ok) break;
          mma_commit_if(lead, &bar_empty[sb]);
          pending = live;
          if (ALONE) pending_b = j & 1;
          pending_first = j == 0;
          pending_last = last;
          ++stage;
        }
        if (tiles == 0) break;
      }
      // every MMA of this warp is complete before TMEM is given back
      mma_commit_if(lead, bar_done);
      mbar_wait<true>(bar_done, 0, nullptr, a.status, 1005);
      __syncwarp();
    } else if (warp < 4) {
      // ---------------------------------------------------------------- Q, rows of both tiles for each of warps 1-3
      constexpr int CHUNKS = D / 8, ROWS = 32 / CHUNKS, STEP = 3 * ROWS;   // 16-byte chunks of a row, rows of a load, of a step
      const int chunk = lane % CHUNKS, r0 = (warp - 1) * ROWS + lane / CHUNKS;
      // elements from a row to the one STEP rows on, and what there is to add where that passes the last head
      const int tokens = STEP / a.G, heads = STEP % a.G;
      const long long by_token = (long long)(a.layout ? a.Hq : 1) * D, by_head = (long long)(a.layout ? 1 : a.Sq) * D;
      const long long on_by = tokens * by_token + heads * by_head, over = by_token - a.G * by_head;
      const uint32_t place = (chunk >> 3) * L::kBoxBytes;
      int loads0 = 0, loads1 = 0;   // of each tile so far
      bool ok = true;
      auto load = [&](const Piece& x, int t, int& loads) {
        const int rows = x.rows - t * kBM;
        if (rows <= 0) return false;
        if (loads > 0 && !(ok = __all_sync(0xffffffffu, mbar_wait<true>(&bar_read[t], (loads - 1) & 1, abort_flag, a.status, 1011)))) return false;
        ++loads;
        const int row = x.unit * kUnit + t * kBM + r0;
        int head = row % a.G;
        const __nv_bfloat16* src = a.q + ((size_t)x.b * a.Hq * a.Sq) * D + (row / a.G) * by_token + (x.h * a.G + head) * by_head + 8 * chunk;
        const uint32_t box = sQ + t * L::kTileBytes + place;
#pragma unroll 2
        for (int r = r0; r < kBM; r += STEP) {   // rows behind the last are zeros
          const bool on = r < rows;
          asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(box + r * 128 + (((chunk & 7) ^ (r & 7)) << 4)),
                       "l"(on ? src : a.q), "r"(on ? 16 : 0) : "memory");
          src += on_by;
          head += heads;
          if (head >= a.G) {
            head -= a.G;
            src += over;
          }
        }
        return true;
      };
      auto there = [&](int t) {
        if (a.q_xor != 0u || a.q_and != 0xffffffffu) {   // a scale that is not positive: this lane's own chunks again
          for (int r = r0; r < kBM; r += STEP) {
            const uint32_t at = sQ + t * L::kTileBytes + place + r * 128 + (((chunk & 7) ^ (r & 7)) << 4);
            const float4 f = ld_shared_f4(at);
            st_shared_v4(at, (__float_as_uint(f.x) & a.q_and) ^ a.q_xor, (__float_as_uint(f.y) & a.q_and) ^ a.q_xor,
                         (__float_as_uint(f.z) & a.q_and) ^ a.q_xor, (__float_as_uint(f.w) & a.q_and) ^ a.q_xor);
          }
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bar_q[t]);
      };
      for (int part = 0; ok; ++part) {
        if (!__all_sync(0xffffffffu, part_there(part))) break;
        const Piece x = pieces[part % kPieces];
        __syncwarp();
        if (lane == 0) mbar_arrive(&bar_past[part % kPieces]);
        if (x.tiles == 0) break;
        load(x, 0, loads0);
        asm volatile("cp.async.commit_group;" ::: "memory");
        const bool both = ok && load(x, 1, loads1);
        asm volatile("cp.async.commit_group;\n\tcp.async.wait_group 1;" ::: "memory");
        if (ok) there(0);
        asm volatile("cp.async.wait_group 0;" ::: "memory");
        if (both) there(1);
      }
    } else {
      // ------------------------------------------------------------------ K and V: from bytes to operands
      const int run = warp - 4;
      int part = 0, left = 0, key = 0, b = 0, h = 0, len = 0;   // of the part: tiles to come, and this warp's first key of the next
      int entries = 0, ahead = 0;   // pages: lane i has the table's entry for this run of the i-th tile of 32, counted down
      // The next tile of the stream, its page's number on its way; false behind the last.
      auto next_tile = [&]() -> bool {
        if (left == 0) {
          if (!__all_sync(0xffffffffu, part_there(part))) return false;
          const Piece& x = pieces[part % kPieces];
          left = x.tiles;
          key = x.tile * kBN + kRun * run - kBN;
          b = x.b;
          h = x.h;
          len = x.len;
          __syncwarp();
          if (lane == 0) mbar_arrive(&bar_past[part % kPieces]);
          ++part;
          if (left == 0) return false;
          ahead = 0;
        }
        key += kBN;
        --left;
        if constexpr (PAGED) {
          if (--ahead < 0) {
            ahead = 31;
            const int mine = key + lane * kBN;
            if (mine < len && lane <= left) entries = __ldg(a.pages.table + b * a.pages.stride + page_index(a.pages, mine));
          }
        }
        return true;
      };
      // Where its run lies.
      auto row_of_tile = [&]() -> long long {
        if constexpr (!PAGED) return ((long long)b * a.c.Hkv + h) * a.c.S + key;
        const int page = __shfl_sync(0xffffffffu, entries, 31 - ahead);
        return key < len ? row_in_page(a.pages, page, a.c.Hkv, h, key, lane == 0 ? a.status : nullptr) : -1;
      };
      RunBytes<D, Q4> k, v;
      long long row = 0;
      int keys = 0;
      bool has_k = next_tile(), has_v = false;
      if (has_k) {
        row = row_of_tile();
        keys = len - key;
        k.load(a.c.k_q, a.c.k_d, row, keys);
      }
      for (int stage = 0; has_k || has_v; ++stage) {
        // K of a tile is on its way, and V of the one before it if there is one
        const int sb = stage % L::kStages;
        const bool more = has_k && next_tile();
        if (stage >= L::kStages &&
            !__all_sync(0xffffffffu, mbar_wait<true>(&bar_empty[sb], (stage / L::kStages - 1) & 1, abort_flag, a.status, 1006)))
          break;
        const uint32_t at = sKV + 2 * sb * L::kTileBytes;
        long long next_row = 0;
        int next_keys = 0;
        if (has_k) {
          k.store(at, run, false);
          if (more) {
            next_row = row_of_tile();
            next_keys = len - key;
            k.load(a.c.k_q, a.c.k_d, next_row, next_keys);
          }
        }
        if (has_v) v.store(at + L::kTileBytes, run, true);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bar_full[sb]);
        if (has_k) v.load(a.c.v_q, a.c.v_d, row, keys);
        has_v = has_k;
        has_k = more;
        row = next_row;
        keys = next_keys;
      }
    }
  } else {
    regs_inc<kRegsSoftmax>();
    // ------------------------------------------------------------------ softmax, a row for each thread
    const int t = (warp - 12) / 4, wq = warp & 3;
    const int r = wq * 32 + lane;   // row of the tile
    const uint32_t lane_off = (uint32_t)(wq * 32) << 16;
    uint32_t tS = tmem + t * 128 + lane_off;   // ALONE: of the buffer at hand
    const uint32_t tO = tmem + 256 + t * D + lane_off;
    const float sl2 = a.sl2;
    // the next part with live rows in this tile of rows, from part `i` on; false behind the last
    auto next_live = [&](int& i) -> bool {
      for (;; ++i) {
        if (!__all_sync(0xffffffffu, part_there(i))) return false;
        const Piece& x = pieces[i % kPieces];
        const int rows = x.rows, tiles = x.tiles;
        if (tiles != 0 && rows > t * kBM) return true;
        if (tiles == 0) return false;
        __syncwarp();
        if (lane == 0) mbar_arrive(&bar_past[i % kPieces]);
      }
    };
    bool ok = true;
    int scored = 0, finished = 0;   // completions of bar_s and bar_o so far
    int b = t, scored1 = 0, made = 0;   // ALONE: the buffer at hand; of bar_s[1]; products of weights that are there, done or to come
    int part = 0;
    for (; next_live(part); ++part) {
      int key0, key_hi, left;   // of the next tile: its first key, and the last one that this row sees
      {
        const Piece& x = pieces[part % kPieces];
        const bool live = t * kBM + r < x.rows;
        key0 = x.tile * kBN;
        key_hi = live ? x.len - x.n + (x.unit * kUnit + t * kBM + r) / a.G : -1;
        left = x.tiles;
      }
      const int key_lo = a.window > 0 ? key_hi - a.window : 0;
      float m = -CUDART_INF_F, l = 0.f;
      bool first = true;
      if constexpr (ALONE) {
        b = 0;
        tS = tmem + lane_off;
      }
      for (; left > 0; --left, key0 += kBN, first = false) {
        if (!(ok = __all_sync(0xffffffffu, mbar_wait<true>(&bar_s[b], (ALONE && b ? scored1 : scored) & 1, abort_flag, a.status, 1007)))) break;
        if (ALONE && b) ++scored1;
        else ++scored;
        tc_fence_after();
        const int lo = min(max(key_lo - key0, 0), kBN), lim = max(min(key_hi - key0, kBN - 1), -1);
        const bool full = lo == 0 && lim == kBN - 1;
        // scores 32 c .. of the row, hidden ones -inf
        auto masked = [&](uint32_t (&x)[32], int c) {
          if (full) return;
          const int from = max(lo - 32 * c, 0), to = min(lim - 32 * c + 1, 32);
          const uint32_t seen = to <= from ? 0u : (uint32_t)(((1ull << to) - 1ull) & ~((1ull << from) - 1ull));
#pragma unroll
          for (int e = 0; e < 32; ++e) x[e] = (seen >> e) & 1u ? x[e] : 0xff800000u;
        };
        const uint64_t sl2_2 = f32x2(sl2, sl2);
        uint64_t sum2[2] = {f32x2(0.f, 0.f), f32x2(0.f, 0.f)};
#pragma unroll 1
        for (int c = 0; c < kBN / 32; ++c) {   // rolled, like the loaders: what warps go through has to come from the instruction caches
          uint32_t x[32];
          tmem_ld32(tS + c * 32, x);
          tmem_wait_ld();
          reg_fence(x);
          masked(x, c);
          float top2[2] = {-CUDART_INF_F, -CUDART_INF_F};
#pragma unroll
          for (int e = 0; e < 32; e += 2) top2[(e >> 1) & 1] = max3f(top2[(e >> 1) & 1], __uint_as_float(x[e]), __uint_as_float(x[e + 1]));
          const float top = fmaxf(top2[0], top2[1]) * sl2;
          if (__any_sync(0xffffffffu, top > m + kRescale)) {   // rare, but for a unit's first scores
            // a whole number: what there is changes by a power of two, so nothing is rounded again
            const float m_new = top > m + kRescale ? ceilf(top) : m;
            const float alpha = m_new == m ? 1.f : ex2_approx(m - m_new);
            m = m_new;
            l *= alpha;
            const uint64_t alpha_2 = f32x2(alpha, alpha);
            sum2[0] = mul_f32x2(sum2[0], alpha_2);
            sum2[1] = mul_f32x2(sum2[1], alpha_2);
            const uint32_t alpha_16 = pack_bf16x2(alpha, alpha);
            tmem_wait_st();
#pragma unroll 1
            for (int d = 0; d < c; ++d) {   // weights of this tile that are stored already
              uint32_t pk[16];
              tmem_ld16(tS + d * 16, pk);
              tmem_wait_ld();
              reg_fence16(pk);
#pragma unroll
              for (int e = 0; e < 16; ++e) pk[e] = mul_bf16x2(pk[e], alpha_16);
              tmem_st16(tS + d * 16, pk);
            }
            if (!first) {   // O holds the products of the tiles before: their MMAs ended before these scores did
              if constexpr (ALONE) {   // ... but for the last one's, product made - 1; what a wait has seen passes at once again
                const bool there = mbar_wait<true>(&bar_v[(made - 1) & 1], ((made - 1) >> 1) & 1, abort_flag, a.status, 1012);
                ok = __all_sync(0xffffffffu, there) && ok;
                tc_fence_after();
              }
#pragma unroll 1
              for (int d = 0; d < D / 16; ++d) {
                uint32_t ov[16];
                tmem_ld16(tO + d * 16, ov);
                tmem_wait_ld();
                reg_fence16(ov);
#pragma unroll
                for (int e = 0; e < 16; ++e) ov[e] = __float_as_uint(__uint_as_float(ov[e]) * alpha);
                tmem_st16(tO + d * 16, ov);
              }
            }
          }
          const float less = m == -CUDART_INF_F ? 0.f : -m;
          const uint64_t less_2 = f32x2(less, less);
          uint32_t pk[16];
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            float t0, t1;
            f32x2_split(fma_f32x2(f32x2(__uint_as_float(x[2 * e]), __uint_as_float(x[2 * e + 1])), sl2_2, less_2), t0, t1);
            const float p0 = ex2_approx(t0), p1 = ex2_approx(t1);
            sum2[e & 1] = add_f32x2(sum2[e & 1], f32x2(p0, p1));
            pk[e] = pack_bf16x2(p0, p1);
          }
          tmem_st16(tS + c * 16, pk);   // over scores that have been read
        }
        float s0, s1, s2, s3;
        f32x2_split(sum2[0], s0, s1);
        f32x2_split(sum2[1], s2, s3);
        l += (s0 + s1) + (s2 + s3);
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bar_p[b]);
        if constexpr (ALONE) {
          if (!ok) break;
          ++made;
          b ^= 1;
          tS = tmem + b * 128 + lane_off;
        }
      }
      if (!ok) break;
      if (!(ok = __all_sync(0xffffffffu, mbar_wait<true>(&bar_o[t], finished & 1, abort_flag, a.status, 1008)))) break;
      ++finished;
      tc_fence_after();
      const Piece& x = pieces[part % kPieces];
      const bool live = t * kBM + r < x.rows, whole = x.starts && x.ends;
      const RowPlace place = place_of(a, x.b, x.h, live ? x.unit * kUnit + t * kBM + r : 0);
      const bool alive = l != 0.f;   // a sum that is no number is one
      const float inv = !whole ? 1.f : alive ? 1.f / l : 0.f;
      uint4* out = reinterpret_cast<uint4*>(a.o + place.at);
      const size_t slot = ((size_t)blockIdx.x * 2 + (x.starts ? 1 : 0)) * a.part_rows + t * kBM + r;
      uint4* left_o = reinterpret_cast<uint4*>(a.part_o + slot * D);
#pragma unroll
      for (int cch = 0; cch < D / 32; ++cch) {
        uint32_t ov[32];
        tmem_ld32(tO + cch * 32, ov);
        tmem_wait_ld();
        reg_fence(ov);
        if (!live) continue;
        float f[32];
#pragma unroll
        for (int e = 0; e < 32; ++e) f[e] = alive ? __uint_as_float(ov[e]) * inv : 0.f;
        if (whole) {
#pragma unroll
          for (int e = 0; e < 2; ++e)
            st_global_32(a.wide, out + cch * 4 + 2 * e, pack_bf16x2(f[16 * e], f[16 * e + 1]), pack_bf16x2(f[16 * e + 2], f[16 * e + 3]),
                         pack_bf16x2(f[16 * e + 4], f[16 * e + 5]), pack_bf16x2(f[16 * e + 6], f[16 * e + 7]),
                         pack_bf16x2(f[16 * e + 8], f[16 * e + 9]), pack_bf16x2(f[16 * e + 10], f[16 * e + 11]),
                         pack_bf16x2(f[16 * e + 12], f[16 * e + 13]), pack_bf16x2(f[16 * e + 14], f[16 * e + 15]));
        } else {
#pragma unroll
          for (int e = 0; e < 4; ++e)
            st_global_32(true, left_o + cch * 8 + 2 * e, __float_as_uint(f[8 * e]), __float_as_uint(f[8 * e + 1]), __float_as_uint(f[8 * e + 2]),
                         __float_as_uint(f[8 * e + 3]), __float_as_uint(f[8 * e + 4]), __float_as_uint(f[8 * e + 5]),
                         __float_as_uint(f[8 * e + 6]), __float_as_uint(f[8 * e + 7]));
        }
      }
      tc_fence_before();   // these reads of O come before the next part's product, which waits for bar_p
      if (live) {
        if (whole) a.lse[place.log] = alive ? (m + log2f(l)) * kLn2 : 0.f;
        else a.part_ml[slot] = make_float2(alive ? m : -CUDART_INF_F, l);
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&bar_past[part % kPieces]);
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 0) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// Joins the parts of the units that slices share: of each row the parts by their weights, in the order of the slices. Units
// of few parts have a warp for each row, of many a block; the rows of all units are one list over the blocks.
template <int D>
__global__ void __launch_bounds__(256) prefill_join_kernel(const __grid_constant__ PrefillArgs a, int slices) {
  constexpr int F = D / 32, kMany = 24;   // features of a lane; parts from which on a row is a block's
  using V = std::conditional_t<F == 4, float4, float2>;
  extern __shared__ __align__(16) Record records[];   // [slices], then first_item
  int* first_item = reinterpret_cast<int*>(records + slices);   // [slices + 1]
  __shared__ float so[8][D];
  __shared__ float2 sml[8];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  wait_for_kernel_before();
  for (int i = threadIdx.x; i < 2 * slices; i += 256) reinterpret_cast<int4*>(records)[i] = reinterpret_cast<const int4*>(a.records)[i];
  __syncthreads();
  if (warp == 0) {   // an item: 32 rows of a unit, four for each warp, or one
    int all = 0;
    for (int c0 = 0; c0 < slices; c0 += 32) {
      int own = 0;
      if (c0 + lane < slices) {
        const Record& rec = records[c0 + lane];
        if (rec.c1 >= 0) own = rec.c1 - rec.c0 + 1 > kMany ? rec.rows : (rec.rows + 31) / 32;
      }
      int x = own;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
      }
      if (c0 + lane < slices) first_item[c0 + lane] = all + x - own;
      all += __shfl_sync(0xffffffffu, x, 31);
    }
    if (lane == 0) first_item[slices] = all;
  }
  __syncthreads();
  const int all = first_item[slices];
  auto add = [](float (&o)[F], float w, const V& v) {
    o[0] = fmaf(w, v.x, o[0]);
    o[1] = fmaf(w, v.y, o[1]);
    if constexpr (F == 4) {
      o[2] = fmaf(w, v.z, o[2]);
      o[3] = fmaf(w, v.w, o[3]);
    }
  };
  auto finish = [&](const Record& rec, int row, const float (&o)[F], float top, float l) {
    const RowPlace place = place_of(a, rec.b, rec.h, rec.unit * kUnit + row);
    const bool alive = l != 0.f;
    const float inv = alive ? 1.f / l : 0.f;
    uint32_t* out = reinterpret_cast<uint32_t*>(a.o + place.at + lane * F);
#pragma unroll
    for (int j = 0; j < F; j += 2) out[j / 2] = pack_bf16x2(o[j] * inv, o[j + 1] * inv);
    if (lane == 0) a.lse[place.log] = alive ? (top + log2f(l)) * kLn2 : 0.f;
  };
  for (int item = blockIdx.x; item < all; item += gridDim.x) {
    int c = 0, past = slices;   // the last record that begins at or before the item (those without items begin where the next do)
    while (past - c > 1) {
      const int mid = (c + past) / 2;
      if (first_item[mid] <= item) c = mid;
      else past = mid;
    }
    const Record& rec = records[c];
    const int parts = rec.c1 - rec.c0 + 1, off = item - first_item[c], rows = rec.rows;
    auto place = [&](int p, int row) { return ((size_t)(rec.c0 + p) * 2 + (p == 0 ? 1 : 0)) * a.part_rows + row; };
    if (parts <= kMany) {   // four rows of a warp side by side, eight parts at a time: lane (part, row) looks at one's reference
      const int row0 = off * 32 + warp * 4;
      const int mine = row0 + (lane & 3);
      float top = -CUDART_INF_F, l = 0.f, o[4][F];
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < F; ++j) o[i][j] = 0.f;
      for (int p0 = 0; p0 < parts && row0 < rows; p0 += 8) {
        const int p = p0 + (lane >> 2);
        const float2 ml = p < parts && mine < rows ? a.part_ml[place(p, mine)] : make_float2(-CUDART_INF_F, 0.f);
        float now = ml.x;
#pragma unroll
        for (int x = 4; x < 32; x <<= 1) now = fmaxf(now, __shfl_xor_sync(0xffffffffu, now, x));
        now = fmaxf(now, top);
        const float ref = now == -CUDART_INF_F ? 0.f : now, back = ex2_approx(top - ref), w = ex2_approx(ml.x - ref);
        float sum = w * ml.y;
#pragma unroll
        for (int x = 4; x < 32; x <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, x);
        top = now;
        l = l * back + sum;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float bi = __shfl_sync(0xffffffffu, back, i);
#pragma unroll
          for (int j = 0; j < F; ++j) o[i][j] *= bi;
        }
        for (int k0 = 0; k0 < 8 && p0 + k0 < parts; k0 += 2) {
          V v[2][4];
#pragma unroll
          for (int k = 0; k < 2; ++k)
#pragma unroll
            for (int i = 0; i < 4; ++i)
              if (p0 + k0 + k < parts && row0 + i < rows) v[k][i] = reinterpret_cast<const V*>(a.part_o + place(p0 + k0 + k, row0 + i) * D)[lane];
#pragma unroll
          for (int k = 0; k < 2; ++k)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const float wi = __shfl_sync(0xffffffffu, w, 4 * (k0 + k) + i);
              if (p0 + k0 + k < parts && row0 + i < rows) add(o[i], wi, v[k][i]);
            }
        }
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float ti = __shfl_sync(0xffffffffu, top, i), li = __shfl_sync(0xffffffffu, l, i);
        if (row0 + i < rows) finish(rec, row0 + i, o[i], ti, li);
      }
      continue;
    }
    // a row for the block: its warps take the parts in turn, 32 at a time, one of them for each lane to look at
    float top = -CUDART_INF_F, l = 0.f, o[F];
#pragma unroll
    for (int j = 0; j < F; ++j) o[j] = 0.f;
    for (int p0 = warp; p0 < parts; p0 += 256) {
      const int n = min(32, (parts - p0 + 7) / 8);
      const float2 ml = lane < n ? a.part_ml[place(p0 + lane * 8, off)] : make_float2(-CUDART_INF_F, 0.f);
      const float now = fmaxf(top, warp_max(ml.x)), ref = now == -CUDART_INF_F ? 0.f : now;
      const float back = ex2_approx(top - ref), w = ex2_approx(ml.x - ref);
      top = now;
      l = l * back + warp_sum(w * ml.y);
#pragma unroll
      for (int j = 0; j < F; ++j) o[j] *= back;
      for (int k0 = 0; k0 < n; k0 += 8) {
        V v[8];
#pragma unroll
        for (int k = 0; k < 8; ++k)
          if (k0 + k < n) v[k] = reinterpret_cast<const V*>(a.part_o + place(p0 + (k0 + k) * 8, off) * D)[lane];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const float wk = __shfl_sync(0xffffffffu, w, (k0 + k) & 31);
          if (k0 + k < n) add(o, wk, v[k]);
        }
      }
    }
    __syncthreads();   // the last item's sums are read
    if (lane == 0) sml[warp] = make_float2(top, l);
#pragma unroll
    for (int j = 0; j < F; ++j) so[warp][lane * F + j] = o[j];
    __syncthreads();
    if (warp != 0) continue;
    const float2 ml = lane < 8 ? sml[lane] : make_float2(-CUDART_INF_F, 0.f);
    top = warp_max(ml.x);
    const float w = ex2_approx(ml.x - (top == -CUDART_INF_F ? 0.f : top));
    l = warp_sum(w * ml.y);
#pragma unroll
    for (int j = 0; j < F; ++j) o[j] = 0.f;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const float wk = __shfl_sync(0xffffffffu, w, k);
#pragma unroll
      for (int j = 0; j < F; ++j) o[j] = fmaf(wk, so[k][lane * F + j], o[j]);
    }
    finish(rec, off, o, top, l);
  }
}

struct PrefillPlan {
  int slices, part_rows;
  size_t part_ml, records, total;   // offsets in the workspace; part_o is at 0
};

PrefillPlan plan_prefill(const fa_prefill_params* p, const CacheView& c) {
  PrefillPlan x{};
  x.slices = sm_count();
  const long long rows = (long long)(p->Hq / c.Hkv) * p->Sq;
  x.part_rows = (int)(rows < kUnit ? rows : kUnit);
  const size_t n = (size_t)x.slices * 2 * x.part_rows;
  x.part_ml = align_up(n * c.D * 4);
  x.records = x.part_ml + align_up(n * 8);
  x.total = x.records + align_up(x.slices * sizeof(Record));
  return x;
}

fa_status check_prefill(const fa_prefill_params* p, const fa_cache* c, const fa_pages* pages, CacheView& held, CacheView& cv,
                        PageView& pv, Span& table) {
  clear_error();
  if (p == nullptr) { set_error("params is NULL"); return FA_ERR_INVALID_ARG; }
  const fa_status st = check_paged(c, pages, held, cv, pv, table);
  return st != FA_OK ? st : check_chunk(p, cv);
}

template <int D, bool Q4, bool PAGED, bool ALONE>
fa_status launch_prefill(const PrefillArgs& a, int slices, cudaStream_t st) {
  constexpr int bytes = PrefillSmem<D>::kBytes;
  static_assert(bytes <= 232448, "shared memory of a block");
  auto kernel = prefill_kernel<D, Q4, PAGED, ALONE>;
  static std::atomic<uint64_t> allowed{0};
  if (allowed.load(std::memory_order_acquire) == 0) {
    const fa_status got = check_split(kernel, "prefill launch", kRegsLaunch);
    if (got != FA_OK) return got;
  }
  const cudaError_t e = allow_shared(kernel, bytes, allowed);
  if (e != cudaSuccess) return cuda_status(e, "prefill launch");
  kernel<<<(unsigned)slices, kThreads, bytes, st>>>(a);
  count_launches(1);
  return cuda_status(cudaGetLastError(), "prefill launch");
}

}  // namespace

fa_status check_chunk(const fa_prefill_params* p, const CacheView& cv) {
  if (p->Hq < 1 || p->Hq > 65535) { set_error("Hq=%d outside [1, 65535]", p->Hq); return FA_ERR_INVALID_ARG; }
  if (p->Hq % cv.Hkv != 0) { set_error("Hq=%d is not a multiple of Hkv=%d", p->Hq, cv.Hkv); return FA_ERR_INVALID_ARG; }
  if (p->Sq < 0 || p->Sq > kMaxSeq) { set_error("Sq=%d outside [0, %d]", p->Sq, kMaxSeq); return FA_ERR_INVALID_ARG; }
  if (p->window < 0) { set_error("window=%d must be >= 0 (0 = no window)", p->window); return FA_ERR_INVALID_ARG; }
  if (p->layout != FA_LAYOUT_BHSD && p->layout != FA_LAYOUT_BSHD) { set_error("layout=%d invalid", p->layout); return FA_ERR_INVALID_ARG; }
  if (!std::isfinite(p->scale)) { set_error("scale is not finite"); return FA_ERR_INVALID_ARG; }
  if (p->reserved != 0) { set_error("reserved field must be 0"); return FA_ERR_INVALID_ARG; }
  if (too_large(cv.B, p->Hq, p->Sq, cv.D)) { set_error("Q would hold more than 2^40 elements"); return FA_ERR_INVALID_ARG; }
  if ((long long)cv.B * p->Hq * p->Sq > 0x7fffffffLL - kUnit) { set_error("too many query rows for one call"); return FA_ERR_UNSUPPORTED; }
  return FA_OK;
}

}  // namespace fa

using namespace fa;

extern "C" {

size_t fa_prefill_workspace_size(const fa_prefill_params* p, const fa_cache* c, const fa_pages* pages) {
  CacheView held, cv;
  PageView pv;
  Span table;
  if (check_prefill(p, c, pages, held, cv, pv, table) != FA_OK || p->Sq == 0) return 0;
  return plan_prefill(p, cv).total;
}

fa_status fa_prefill(const fa_prefill_params* p, const void* q, const fa_cache* c, const fa_pages* pages,
                     const int64_t* lengths, const int64_t* count, void* o, float* lse, void* ws, size_t ws_bytes,
                     void* stream) {
  CacheView held, cv;
  PageView pv;
  Span all[10];
  fa_status st = check_prefill(p, c, pages, held, cv, pv, all[9]);
  if (st != FA_OK) return st;
  const size_t rows = (size_t)cv.B * p->Hq * p->Sq;
  cache_spans(held, all);
  all[4] = {q, rows * cv.D * 2, "q"};
  Span* out = all + 5;
  out[0] = {o, rows * cv.D * 2, "o"};
  out[1] = {lse, rows * 4, "lse"};
  all[7] = {lengths, lengths != nullptr ? (size_t)cv.B * 8 : 0, "lengths"};
  all[8] = {count, count != nullptr ? (size_t)cv.B * 8 : 0, "count"};
  if ((st = check_buffers(all, 5, out, 2)) != FA_OK) return st;
  if ((uintptr_t)lengths % 8 != 0 || (uintptr_t)count % 8 != 0) {
    set_error("lengths and count must be 8-byte aligned"); return FA_ERR_INVALID_ARG;
  }
  if ((st = check_apart(all + 7, 3, out, 2)) != FA_OK) return st;
  if (p->Sq == 0) return FA_OK;
  const PrefillPlan plan = plan_prefill(p, cv);
  if ((st = check_ws(ws, ws_bytes, plan.total, all, 10)) != FA_OK) return st;
  char* w = static_cast<char*>(ws);
  PrefillArgs a{};
  a.pages = pv;
  a.part_o = static_cast<float*>(ws);
  a.part_ml = reinterpret_cast<float2*>(w + plan.part_ml);
  a.records = reinterpret_cast<Record*>(w + plan.records);
  a.part_rows = plan.part_rows;
  if ((a.status = device_status_ptr()) == nullptr) return cuda_status(cudaErrorUnknown, "status word");
  a.sl2 = p->scale == 0.f ? 1.f : fminf(fabsf(p->scale) * kLog2e, FLT_MAX);
  a.q_and = p->scale == 0.f ? 0u : 0xffffffffu;
  a.q_xor = p->scale < 0.f ? 0x80008000u : 0u;
  a.Hq = p->Hq;
  a.Sq = p->Sq;
  a.window = p->window < 2 * kMaxSeq ? p->window : 2 * kMaxSeq;
  a.layout = p->layout;
  a.G = p->Hq / cv.Hkv;
  a.wide = (uintptr_t)o % 32 == 0;
  cudaStream_t cs = (cudaStream_t)stream;
  const size_t per = (size_t)p->Hq * p->Sq;   // rows of a sequence
  for (int b0 = 0; b0 < cv.B; b0 += kListed) {
    a.c = cv;
    a.c.B = cv.B - b0 < kListed ? cv.B - b0 : kListed;
    a.q = static_cast<const __nv_bfloat16*>(q) + b0 * per * cv.D;
    a.o = static_cast<__nv_bfloat16*>(o) + b0 * per * cv.D;
    a.lse = lse + b0 * per;
    a.lengths = lengths != nullptr ? lengths + b0 : nullptr;
    a.count = count != nullptr ? count + b0 : nullptr;
    if (pages != nullptr) {
      a.pages.table = pv.table + b0 * pv.stride;
    } else {   // sequence 0 of this launch
      const size_t keys = (size_t)b0 * cv.Hkv * cv.S;
      a.c.k_q = static_cast<uint8_t*>(cv.k_q) + keys * (cv.q4 ? cv.D / 2 : cv.D);
      a.c.v_q = static_cast<uint8_t*>(cv.v_q) + keys * (cv.q4 ? cv.D / 2 : cv.D);
      a.c.k_d = cv.k_d + keys * (cv.D / 32);
      a.c.v_d = cv.v_d + keys * (cv.D / 32);
    }
    auto go = [&](auto dim, auto q4) {
      constexpr int D = decltype(dim)::value;
      constexpr bool Q4 = decltype(q4)::value;
      if ((long long)a.G * p->Sq <= kBM)
        return pages != nullptr ? launch_prefill<D, Q4, true, true>(a, plan.slices, cs) : launch_prefill<D, Q4, false, true>(a, plan.slices, cs);
      return pages != nullptr ? launch_prefill<D, Q4, true, false>(a, plan.slices, cs) : launch_prefill<D, Q4, false, false>(a, plan.slices, cs);
    };
    using D64 = std::integral_constant<int, 64>;
    using D128 = std::integral_constant<int, 128>;
    if (cv.q4) st = cv.D == 64 ? go(D64{}, std::true_type{}) : go(D128{}, std::true_type{});
    else st = cv.D == 64 ? go(D64{}, std::false_type{}) : go(D128{}, std::false_type{});
    if (st != FA_OK) return st;
    cudaLaunchAttribute at{};
    at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(3 * plan.slices);   // what the SMs hold at a time
    cfg.blockDim = dim3(256);
    cfg.dynamicSmemBytes = plan.slices * sizeof(Record) + (plan.slices + 1) * sizeof(int);
    cfg.stream = cs;
    cfg.attrs = &at;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, cv.D == 64 ? prefill_join_kernel<64> : prefill_join_kernel<128>, a, plan.slices);
    count_launches(1);
    if (e != cudaSuccess) return cuda_status(e, "prefill launch");
  }
  return FA_OK;
}

}  // extern "C"
