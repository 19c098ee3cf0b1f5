// Attention of the newest tokens of every sequence over its quantized cache, read in place
// (fa_decode): the serving form of the op, one to a few tokens per sequence.
//
// Mathematics. With G = Hq / Hkv query heads on a key/value head, the R = G * Sq query rows of one
// head all read the same keys. A block of 32 features of a key is d * n with whole numbers n, so
//     s_j = scale * sum_blocks d_jb <n_jb, q_b>,   o = sum_j sum_blocks (p_j d_jb) n_jb :
// the tensor cores multiply whole numbers, exact as fp16, by q and by p * d, and K's scales never touch
// the 8- or 4-bit data. Scores, softmax statistics and sums are fp32. Query rows are scaled by a power of
// two to the top of fp16's range, where a bf16 value down to 2^-24 of the row's largest is exact; p d_jb is
// formed in fp32 and rounded once to fp16. Weights are relative to a power of two (base 2, `base`) that follows the largest
// p d_jb that a query row has met, not the largest p: a first key that takes most of the weight and has small values
// leaves the others their bits, and so does one large value elsewhere. The largest is at least 2^kSet when base is set
// and at most 2^kMost later, so a weight down to 2^(-14 - kSet), 2^-24, of the largest in its run is off by 2^-11 of its value
// at most, and a smaller one by 2^-35 of the largest (a key whose values are all 0 counts with a scale of 2^-32).
//
// What bounds it: the planes are read once, 144 bytes a key for D = 128 in 4 bits, so HBM; next to
// that the instructions that turn packed bits into operands. Keys are the 16 rows of an
// mma.sync m16n8k16 and query rows its 8 columns: with 4 query rows a head a tcgen05 tile of 128
// rows would be 3% full, and its operands would have to be written to shared memory as 16-bit numbers
// first, four times the bytes that are read.
//
// From bits to operands: ldmatrix hands a lane the packed words of its operand rows, for V with two
// keys side by side (transposed). Masked, the four bits b of two bytes are operands already: as fp16 they
// are b 2^-24 (low nibbles) and b 2^-20 (high ones), exact subnormal numbers; the powers of two are
// taken into q and into the result. Each pair of numbers costs one logic instruction, and each word a
// shift. What the format takes off (8, or 128 in 8 bits) is in the products' starting value for K, a
// multiple of the sum of q over a block; V's numbers get a packed addition, exact and on another pipe than
// the logic, as sums over many keys that hold a large offset would lose bits.
//
// Split: the tiles of 32 keys of all sequences and heads are one list, cut into equal slices, one for
// each block that the SMs hold at a time, and those into one run of tiles for each warp: the end of one
// head, whole heads and the beginning of another. A warp walks its run through its own ring of shared
// memory (cp.async) with a reference for its weights of its own and waits for no other; heads that it shares with its
// block's other warps are joined when all are done, those that blocks share by a second kernel. Where
// every head is a few tiles long a block takes one head, and there is no second kernel (see plan_decode). Beginning with a head (its
// queries, the first tile's way) costs a warp about three tiles' time, which the list counts (64 sequences of 512 to 4096
// keys in 8 bits, 32 heads on 8: 61.0 us without, 58.6 with; 500 of up to 300 keys in 4 bits, 8 on 2: 21.8 and 18.4).
//
// Measured (device time, captured calls over changing inputs), 4 bits, D = 128: 64 sequences of 1024 to 8192 keys, 32 heads
// on 8: 62.3 us, 5.5 TB/s, 81% of the measured copy rate; the loop itself runs at that rate, and what is
// left is the way to the first tile (3.7 us), warps that end before others (2 to 3) and the two joins (4). One sequence of
// 67584 keys, 16 heads on 4: 16.2 us against 5.8 for the bytes; a warp has four or five tiles then, and list, first
// tile and joins are most of it. Four sequences of up to 1000 keys in 8 bits, D = 64: 6.0 us, launch and latencies. (With p and p d
// each rounded to fp16, relative to p alone, these took 61.6, 15.9 and 6.1 us; the alternatives to single choices
// below were measured then.)
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
constexpr int kTile = 32;         // keys a warp takes at a time
constexpr int kMaxListed = 1024;  // sequences whose lengths a block lists
constexpr int kStart = 3;         // tiles' time that a head costs the warp that begins with it, measured
constexpr float kNoBase = -3e38f; // below every score
constexpr float kSet = 10.f;      // the largest weight times scale, base 2, when a row's reference is set,
constexpr float kMost = 14.f;     // and what it may become before the reference is set again; fp16 ends at 16
constexpr float kLn2 = 0.6931471805599453f;

struct DecodeArgs {
  CacheView c;
  const __nv_bfloat16* q;
  __nv_bfloat16* o;
  float* lse;
  const int64_t* lengths;
  // slices only: what blocks leave of heads that they share, two slots a block
  float* part_o;         // [row blocks, blocks, 2, rows, D]: unnormalised
  float2* part_ml;       // [row blocks, blocks, 2, rows]: what the weights are relative to (base 2), and their sum
  float* warp_o;         // what a warp leaves of a head that ends inside its run: as part_o, [row blocks, blocks, warps, rows, D];
  float2* warp_ml;       // not used where shared memory has room for it
  unsigned* status;
  float scale2;          // scale * log2(e)
  int Hq, Sq, window, layout;
  int G, R;              // query heads and rows of a key/value head
};

// The keys a sequence's queries may see: [lo, len), lo on a tile's border.
struct Range { int len, lo; };

__device__ __forceinline__ Range key_range(const DecodeArgs& a, long long n, bool report) {
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

__device__ __forceinline__ long long length_of(const DecodeArgs& a, int b) {
  return a.lengths != nullptr ? __ldg(a.lengths + b) : a.c.S;
}

// Element offset of query row r (head r / Sq of the group, token r % Sq) in q and o.
__device__ __forceinline__ size_t q_offset(const DecodeArgs& a, int b, int h, int r) {
  const int head = h * a.G + r / a.Sq, i = r % a.Sq;
  return (a.layout ? ((size_t)b * a.Sq + i) * a.Hq + head : ((size_t)b * a.Hq + head) * a.Sq + i) * a.c.D;
}

__device__ __forceinline__ float bf16_lo(uint32_t x) { return __uint_as_float(x << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t x) { return __uint_as_float(x & 0xffff0000u); }

__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float log2_fast(float x) {
  float y;
  asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
template <int N>
__device__ __forceinline__ void cp_async_small(uint32_t dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(dst), "l"(src), "n"(N) : "memory");
}
// Zeros, and nothing read, where not `on`.
__device__ __forceinline__ void cp_async16_if(uint32_t dst, const void* src, bool on) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(on ? 16 : 0) : "memory");
}
template <int N>
__device__ __forceinline__ void cp_async_small_if(uint32_t dst, const void* src, bool on) {
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
// Kept where it is among the copies.
__device__ __forceinline__ uint2 ld_global64(const void* p) {
  uint2 v;
  asm volatile("ld.global.nc.v2.b32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "l"(p));
  return v;
}
// Four 8 x 8 matrices of 16-bit elements, lane i naming row i % 8 of matrix i / 8: of matrix j lane
// (g, t) gets elements 2 t, 2 t + 1 of row g, or, transposed, element g of rows 2 t and 2 t + 1.
template <bool TRANS>
__device__ __forceinline__ void load_matrices(uint32_t at, uint32_t (&x)[4]) {
  if constexpr (TRANS)
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(x[0]), "=r"(x[1]), "=r"(x[2]), "=r"(x[3]) : "r"(at) : "memory");
  else
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(x[0]), "=r"(x[1]), "=r"(x[2]), "=r"(x[3]) : "r"(at) : "memory");
}

__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// From other values than the result's: c0 and c1 in both rows.
__device__ __forceinline__ void mma_f16_from(float (&d)[4], float c0, float c1, uint32_t a0, uint32_t a1, uint32_t a2,
                                             uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%11,%10,%11};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(c0), "f"(c1));
}

__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  const __half2 r = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&r);
}

__device__ __forceinline__ uint32_t add_f16x2(uint32_t x, uint32_t y) {
  const __half2 r = __hadd2(*reinterpret_cast<const __half2*>(&x), *reinterpret_cast<const __half2*>(&y));
  return *reinterpret_cast<const uint32_t*>(&r);
}

// Fp16 operands, numbers times 2^-24, from the packed words of a block. 4 bits, one word: the numbers of
// bytes (0, 2) and (1, 3), first those of the low nibbles, then, 16 times as large, of the high ones.
__device__ __forceinline__ void pairs_q4(uint32_t w, uint32_t (&f)[4]) {
  const uint32_t h = w >> 8;
  f[0] = w & 0x000f000fu;
  f[1] = h & 0x000f000fu;
  f[2] = w & 0x00f000f0u;
  f[3] = h & 0x00f000f0u;
}
// 8 bits, one word of each half block, numbers + 128: bytes (A, B) and (C, D) of the first, then of the second.
template <int A, int B, int C, int D>
__device__ __forceinline__ void pairs_q8(uint32_t w0, uint32_t w1, uint32_t (&f)[4]) {
  const uint32_t a = w0 ^ 0x80808080u, b = w1 ^ 0x80808080u;
  f[0] = __byte_perm(a, 0u, 0x4040 | A | B << 8);
  f[1] = __byte_perm(a, 0u, 0x4040 | C | D << 8);
  f[2] = __byte_perm(b, 0u, 0x4040 | A | B << 8);
  f[3] = __byte_perm(b, 0u, 0x4040 | C | D << 8);
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
  static constexpr int STAGES = 2;                // 3 measured no faster
  // Piece p of a row is at piece p ^ (row / PER) % PIECES, PER the rows in 128 bytes: the rows of a
  // matrix then meet no bank twice. Rows 8 apart are permuted alike.
  static constexpr int PER = 128 / ROW;
  __device__ static __forceinline__ int permuted(unsigned row) { return (int)(row / PER % PIECES); }
};

// The scales of a key.
template <int NB>
__device__ __forceinline__ void load_scales(uint32_t at, float (&d)[NB]) {
  uint32_t u[NB / 2];
  if constexpr (NB == 4) {
    const uint2 x = lds64(at);
    u[0] = x.x; u[1] = x.y;
  } else {
    u[0] = lds32(at);
  }
#pragma unroll
  for (int i = 0; i < NB / 2; ++i) {
    const float2 x = __half22float2(*reinterpret_cast<const __half2*>(&u[i]));
    d[2 * i] = x.x;
    d[2 * i + 1] = x.y;
  }
}
// As they are, two a word.
template <int NB>
__device__ __forceinline__ void load_scale_words(uint32_t at, uint32_t (&u)[NB / 2]) {
  if constexpr (NB == 4) {
    const uint2 x = lds64(at);
    u[0] = x.x; u[1] = x.y;
  } else {
    u[0] = lds32(at);
  }
}
__device__ __forceinline__ float scale_of(uint32_t u, bool high) {
  const __half2 x = *reinterpret_cast<const __half2*>(&u);
  return high ? __high2float(x) : __low2float(x);
}
// The base 2 logarithm of the largest magnitude among a key's scales, held to [-32, 16]: below fp16's smallest where all are
// 0, so that a key without values does not set what the others' weights are relative to.
template <int NB>
__device__ __forceinline__ float log2_largest(const uint32_t (&u)[NB / 2]) {
  __half2 x = __habs2(*reinterpret_cast<const __half2*>(&u[0]));
  if constexpr (NB == 4) x = __hmax2(x, __habs2(*reinterpret_cast<const __half2*>(&u[1])));
  return fminf(fmaxf(log2_fast(__half2float(__hmax(__low2half(x), __high2half(x)))), -32.f), 16.f);
}

// Warps of a block and blocks an SM holds. Rows of 128 features want 168 registers a thread (at 128 they spilled in the
// loop: 64 sequences of up to 8192 keys in 4 bits then took 81 us with 16 warps on an SM and 76 us with 12).
constexpr int warps_of(int D) { return D == 128 ? 4 : 8; }
constexpr int held_of(int D, int nt) { return D == 128 ? (nt == 1 ? 3 : 2) : (nt == 1 ? 2 : 1); }
// Warps of a block that has an SM to itself.
constexpr int wide_of(int D, int nt) { return warps_of(D) * held_of(D, nt); }

// Bytes of what a block's warps leave: [warps][rows][D] and [warps][rows] pairs. One set of it, of the heads that the
// warps' runs end in, takes the rings' place at the end. The other, of the heads that end inside a run, has a place of
// its own where that costs no block on an SM (not beside the rings of 128 features in 8 bits).
constexpr int left_bytes(int warps, int D, int nt) { return warps * nt * 8 * (D * 4 + 8); }
constexpr bool left_in_memory(int D, bool q4, int nt) { return D == 128 && !q4 && nt == 1; }

// `total` units (below 2^30: a tensor has 2^40 elements at most) cut into n slices that differ by one at most, the larger
// ones first.
struct Slices {
  unsigned each, more;
  __device__ __forceinline__ Slices(unsigned total, unsigned n) : each(total / n), more(total % n) {}
  __device__ __forceinline__ unsigned begin(unsigned i) const { return i * each + min(i, more); }
  __device__ __forceinline__ unsigned of(unsigned unit) const {
    const unsigned large = more * (each + 1);
    return unit < large ? unit / (each + 1) : more + (unit - large) / each;
  }
};

// Units of the sequences before each, per key/value head, into list[0 .. B] in shared memory (all threads): a head's tiles, and
// kStart for what it costs a warp to begin with it.
template <int THREADS>
__device__ __forceinline__ void make_list(const DecodeArgs& a, int* list, bool report) {
  constexpr int EACH = (kMaxListed + THREADS - 1) / THREADS;
  __shared__ int warp_sum[THREADS / 32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int each = (a.c.B + THREADS - 1) / THREADS, first = threadIdx.x * each;   // this thread's sequences
  long long length[EACH];
#pragma unroll
  for (int i = 0; i < EACH; ++i) {   // all on their way at once
    if (i >= each) break;
    length[i] = first + i < a.c.B ? length_of(a, first + i) : 0;
  }
  int units[EACH], x = 0;
#pragma unroll
  for (int i = 0; i < EACH; ++i) {
    if (i >= each) break;
    const Range kr = key_range(a, length[i], report);
    const int n = (kr.len - kr.lo + kTile - 1) / kTile;
    units[i] = n > 0 ? n + kStart : 0;
    x += units[i];
  }
  int before = -x;   // less its own: of the threads before this one
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) warp_sum[warp] = x;
  __syncthreads();
  before += x;
#pragma unroll
  for (int w = 0; w < THREADS / 32; ++w)
    if (w < warp) before += warp_sum[w];
#pragma unroll
  for (int i = 0; i < EACH; ++i) {
    if (i >= each) break;
    if (first + i < a.c.B) list[first + i] = before;
    before += units[i];
  }
  if (first < a.c.B && first + each >= a.c.B) list[a.c.B] = before;   // all
  __syncthreads();
}

// The sequence that unit `at` of all heads' is of (all lanes of a warp, one answer): the last that begins at or before it.
__device__ __forceinline__ int sequence_of(const int* list, int B, unsigned heads, unsigned at) {
  const int lane = threadIdx.x & 31, step = (B + 31) / 32;
  const int far = lane * step;
  int b = (__popc(__ballot_sync(0xffffffffu, far < B && list[min(far, B)] * heads <= at)) - 1) * step;
  if (step > 1) {
    const int near = b + lane;
    b += __popc(__ballot_sync(0xffffffffu, lane < step && near < B && list[min(near, B)] * heads <= at)) - 1;
  }
  return b;
}

// A part of a row's sums, by its weight.
__device__ __forceinline__ void add_part(float (&o)[2], float w, float2 x) {
  o[0] = fmaf(w, x.x, o[0]);
  o[1] = fmaf(w, x.y, o[1]);
}
__device__ __forceinline__ void add_part(float (&o)[4], float w, float4 x) {
  o[0] = fmaf(w, x.x, o[0]);
  o[1] = fmaf(w, x.y, o[1]);
  o[2] = fmaf(w, x.z, o[2]);
  o[3] = fmaf(w, x.w, o[3]);
}

// (base + log2 l) ln 2, l's power of two added first: base is about its negative where the logarithm is small.
__device__ __forceinline__ float lse_of(float base, float l) {
  int e;
  const float m = frexpf(l, &e);
  return (base + (float)e + log2f(m)) * kLn2;
}

// Row r of a head from a warp's sums (D / 32 features a lane): the result, or what is left of it.
template <int D>
__device__ __forceinline__ void store_row(const DecodeArgs& a, int b, int h, int r, const float (&o)[D / 32], float l,
                                          float top, bool whole, float* part_o, float2* part_ml) {
  constexpr int F = D / 32;
  const int lane = threadIdx.x & 31;
  if (!whole) {
    if constexpr (F == 4) reinterpret_cast<float4*>(part_o)[lane] = make_float4(o[0], o[1], o[2], o[3]);
    else reinterpret_cast<float2*>(part_o)[lane] = make_float2(o[0], o[1]);
    if (lane == 0) *part_ml = make_float2(top, l);
    return;
  }
  const float inv = l == 0.f ? 0.f : 1.f / l;
  uint32_t* dst = reinterpret_cast<uint32_t*>(a.o + q_offset(a, b, h, r) + lane * F);
#pragma unroll
  for (int j = 0; j < F; j += 2) dst[j / 2] = tc::pack_bf16x2(o[j] * inv, o[j + 1] * inv);
  if (lane == 0) a.lse[((size_t)b * a.Hq + h * a.G) * a.Sq + r] = l == 0.f ? 0.f : lse_of(top, l);
}

// A block's work: SLICES: slice blockIdx.x of the list; else the head blockIdx.x. NT * 8 query rows from
// blockIdx.y * NT * 8 on.
template <int D, bool Q4, int NT, bool SLICES, int kWarps>
__global__ void __launch_bounds__(kWarps * 32, kWarps == warps_of(D) ? held_of(D, NT) : 1) decode_kernel(DecodeArgs a) {
  using S = Slot<D, Q4>;
  constexpr int NB = S::NB, ROWS = NT * 8;
  using V = std::conditional_t<D == 128, float4, float2>;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ int list[SLICES ? kMaxListed + 1 : 1];
  // the heads whose sums the block's warps leave unfinished, in the order of their tiles: two for each
  // warp, the one its run begins in and the one it ends in (-1: none), and how many tiles they had
  __shared__ int left_head[2 * kWarps], left_tiles[2 * kWarps];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int g = lane >> 2, t = lane & 3;
  const int r0 = blockIdx.y * ROWS;
  const uint32_t ring = tc::smem_u32(smem) + warp * (S::STAGES * S::BYTES);
  const bool report = r0 == 0 && (!SLICES || blockIdx.x == 0);
  if constexpr (SLICES) let_next_kernel_start();
  // the matrix row that this lane names: key `lane` of a tile
  const uint32_t mrow = lane * S::ROW;
  const int mperm = S::permuted(lane);
  // -8 or -128 as fp16 in the units of the first and of the second half of a block: subnormal, minus 8, 128 or 128 steps
  constexpr uint32_t kOff0 = Q4 ? 0x80088008u : 0x80808080u, kOff1 = 0x80808080u;

  float acc[NT][2 * NB][4];   // rows: features 16 i + 2 g (and + 1); columns: query rows 2 t, 2 t + 1
  float base[NT][2];          // weights are 2^(score - base)
  float sum[NT][2];           // of this lane's weights

  // The sums over tiles [first_tile, first_tile + tiles) of one head.
  auto run = [&](int b, int h, const Range kr, int first_tile, int tiles) {
    const int k0 = kr.lo + first_tile * kTile;
    // lane's part of a tile's loads: pieces lane, lane + 32, ... of the numbers, key `lane`'s scales
    const unsigned lrow = (unsigned)lane / S::PIECES;
    const int lpiece = lane % S::PIECES;
    const size_t begin = ((size_t)b * a.c.Hkv + h) * a.c.S + k0;
    const uint8_t* kq = static_cast<const uint8_t*>(a.c.k_q) + begin * S::ROW + 16 * lane;
    const uint8_t* vq = static_cast<const uint8_t*>(a.c.v_q) + begin * S::ROW + 16 * lane;
    const uint16_t* kd = a.c.k_d + (begin + lane) * NB;
    const uint16_t* vd = a.c.v_d + (begin + lane) * NB;
    int loaded = k0;   // the first key of the next tile to load
    auto load = [&](uint32_t at) {
      if (loaded + kTile <= kr.len) {
#pragma unroll
        for (int i = 0; i < S::PIECES; ++i) {
          const unsigned row = lrow + i * (32 / S::PIECES);
          const uint32_t dst = at + row * S::ROW + 16 * (lpiece ^ S::permuted(row));
          cp_async16(dst, kq + 512 * i);
          cp_async16(dst + S::V_OFF, vq + 512 * i);
        }
        cp_async_small<S::SC>(at + S::KD_OFF + lane * S::SC, kd);
        cp_async_small<S::SC>(at + S::VD_OFF + lane * S::SC, vd);
      } else {   // the last tile: keys past the end are zeros, and not read
#pragma unroll
        for (int i = 0; i < S::PIECES; ++i) {
          const unsigned row = lrow + i * (32 / S::PIECES);
          const uint32_t dst = at + row * S::ROW + 16 * (lpiece ^ S::permuted(row));
          const bool on = loaded + (int)row < kr.len;
          cp_async16_if(dst, on ? kq + 512 * i : static_cast<const uint8_t*>(a.c.k_q), on);
          cp_async16_if(dst + S::V_OFF, on ? vq + 512 * i : static_cast<const uint8_t*>(a.c.v_q), on);
        }
        const bool on = loaded + lane < kr.len;
        cp_async_small_if<S::SC>(at + S::KD_OFF + lane * S::SC, on ? kd : a.c.k_d, on);
        cp_async_small_if<S::SC>(at + S::VD_OFF + lane * S::SC, on ? vd : a.c.v_d, on);
      }
      loaded += kTile;
      kq += kTile * S::ROW;
      vq += kTile * S::ROW;
      kd += kTile * NB;
      vd += kTile * NB;
    };
    auto commit = [] { asm volatile("cp.async.commit_group;" ::: "memory"); };

    // the query rows on their way before the tiles that would hold them up: of row g of each eight the features
    // 4 t .. 4 t + 3 of every half block
    uint2 raw[NT][NB][2];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const int r = r0 + n * 8 + g;
      const __nv_bfloat16* src = a.q + (r < a.R ? q_offset(a, b, h, r) : 0) + 4 * t;
#pragma unroll
      for (int k = 0; k < NB; ++k)
#pragma unroll
        for (int st = 0; st < 2; ++st) {
          raw[n][k][st] = make_uint2(0, 0);
          if (r < a.R) raw[n][k][st] = ld_global64(src + 32 * k + 16 * st);
        }
    }
#pragma unroll
    for (int i = 0; i < S::STAGES - 1; ++i) {
      if (i < tiles) load(ring + i * S::BYTES);
      commit();
    }

    // the query rows as operands: lane (g, t) holds, of row g, the features whose numbers its words
    // of a key's block hold; each row by a power of two at the top of fp16's range, with the softmax
    // scale's sign
    uint32_t qf[NT][NB][2][2];
    float bias[NT][NB][2];  // what the numbers' offset makes of a block's q, of columns 2 t and 2 t + 1
    float unscale[NT][2];   // scores in base 2, of columns 2 t and 2 t + 1: the products by this; not negative
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      float top = 0.f;
#pragma unroll
      for (int k = 0; k < NB; ++k)
#pragma unroll
        for (int st = 0; st < 2; ++st) {
          const uint2 x = raw[n][k][st];
          top = fmaxf(top, fmaxf(fmaxf(fabsf(bf16_lo(x.x)), fabsf(bf16_hi(x.x))), fmaxf(fabsf(bf16_lo(x.y)), fabsf(bf16_hi(x.y)))));
        }
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
      // 2^(14 - e) for a top in [2^e, 2^(e + 1)); exponents held to what 2^x and its inverse have room for
      const int e = (int)(__float_as_uint(top) >> 23) - 127;
      const int up = top > 0.f && e < 128 ? max(min(14 - e, 126), -100) : 0;
      const float f = copysignf(__uint_as_float((uint32_t)(127 + up) << 23), a.scale2);
      const float back = __uint_as_float((uint32_t)(127 + 24 - up) << 23) * fabsf(a.scale2);
#pragma unroll
      for (int k = 0; k < NB; ++k) {
        float q_sum = 0.f;
#pragma unroll
        for (int st = 0; st < 2; ++st) {
          const float x0 = bf16_lo(raw[n][k][st].x) * f, x1 = bf16_hi(raw[n][k][st].x) * f;
          const float x2 = bf16_lo(raw[n][k][st].y) * f, x3 = bf16_hi(raw[n][k][st].y) * f;
          q_sum += (x0 + x1) + (x2 + x3);
          const float down = Q4 && st == 1 ? 1.f / 16 : 1.f;   // high nibbles are 16 times as large
          qf[n][k][st][0] = Q4 ? pack_f16x2(x0 * down, x2 * down) : pack_f16x2(x0, x1);
          qf[n][k][st][1] = Q4 ? pack_f16x2(x1 * down, x3 * down) : pack_f16x2(x2, x3);
        }
        q_sum += __shfl_xor_sync(0xffffffffu, q_sum, 1);
        q_sum += __shfl_xor_sync(0xffffffffu, q_sum, 2);
        q_sum *= Q4 ? -8.f / 16777216 : -128.f / 16777216;
        bias[n][k][0] = __shfl_sync(0xffffffffu, q_sum, 8 * t);
        bias[n][k][1] = __shfl_sync(0xffffffffu, q_sum, 8 * t + 4);
      }
      unscale[n][0] = __shfl_sync(0xffffffffu, back, 8 * t);
      unscale[n][1] = __shfl_sync(0xffffffffu, back, 8 * t + 4);
    }

#pragma unroll
    for (int n = 0; n < NT; ++n) {
#pragma unroll
      for (int i = 0; i < 2 * NB; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[n][i][j] = 0.f;
      base[n][0] = base[n][1] = kNoBase;
      sum[n][0] = sum[n][1] = 0.f;
    }
    // keys that every query row sees: [all_from, all_to]
    const int all_to = kr.len - a.Sq, all_from = a.window > 0 ? kr.len - 1 - a.window : 0;

    // One tile, in the ring at `at`, from key `first` on. EDGE: some query row does not see all of it.
    auto step = [&](auto on_edge, uint32_t at, int first) {
      constexpr bool EDGE = decltype(on_edge)::value;
      // products of 2 x 16 keys
      float s[NT][2][4];
      float d[4][NB];   // K's scales, of keys g, g + 8, g + 16, g + 24
#pragma unroll
      for (int i = 0; i < 4; ++i) load_scales<NB>(at + S::KD_OFF + (8 * i + g) * S::SC, d[i]);
#pragma unroll
      for (int k = 0; k < NB; ++k) {
        uint32_t f[4][4];   // [keys 8 i ..][pairs]
        if constexpr (Q4) {
          uint32_t w[4];
          load_matrices<false>(at + mrow + 16 * (k ^ mperm), w);
#pragma unroll
          for (int i = 0; i < 4; ++i) pairs_q4(w[i], f[i]);
        } else {
          uint32_t w[4], x[4];
          load_matrices<false>(at + mrow + 16 * ((2 * k) ^ mperm), w);
          load_matrices<false>(at + mrow + 16 * ((2 * k + 1) ^ mperm), x);
#pragma unroll
          for (int i = 0; i < 4; ++i) pairs_q8<0, 1, 2, 3>(w[i], x[i], f[i]);
        }
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int m = 0; m < 2; ++m) {
            float c[4];
            mma_f16_from(c, bias[n][k][0], bias[n][k][1], f[2 * m][0], f[2 * m + 1][0], f[2 * m][1], f[2 * m + 1][1],
                         qf[n][k][0][0], qf[n][k][0][1]);
            mma_f16(c, f[2 * m][2], f[2 * m + 1][2], f[2 * m][3], f[2 * m + 1][3], qf[n][k][1][0], qf[n][k][1][1]);
#pragma unroll
            for (int j = 0; j < 4; j += 2) {   // a key's two columns, packed
              const uint64_t dd = tc::f32x2(d[2 * m + j / 2][k], d[2 * m + j / 2][k]), cc = tc::f32x2(c[j], c[j + 1]);
              tc::f32x2_split(k == 0 ? tc::mul_f32x2(dd, cc) : tc::fma_f32x2(dd, cc, tc::f32x2(s[n][m][j], s[n][m][j + 1])),
                              s[n][m][j], s[n][m][j + 1]);
            }
          }
      }

      // V's scales, of the same keys
      uint32_t dv[4][NB / 2];
      float lg[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        load_scale_words<NB>(at + S::VD_OFF + (8 * i + g) * S::SC, dv[i]);
        lg[i] = log2_largest<NB>(dv[i]);
      }

      uint32_t hidden[NT];   // bit 2 i + j: of key 8 i + g and column 2 t + j
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        hidden[n] = 0;
        if constexpr (EDGE) {
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const int pos = kr.len - a.Sq + (r0 + n * 8 + 2 * t + j) % a.Sq;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const int key = first + 8 * i + g;
              if (key > pos || (a.window > 0 && pos - key > a.window)) {
                s[n][i / 2][i % 2 * 2 + j] = -CUDART_INF_F;
                hidden[n] |= 1u << (2 * i + j);
              }
            }
          }
        }
        float top[2];   // of p d, base 2
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          float x[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) x[i] = fmaf(s[n][i / 2][i % 2 * 2 + j], unscale[n][j], lg[i]);
          top[j] = fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3]));
        }
        // The reference stays until a weight times its scale outgrows it, which no lane has to ask the others for.
        const bool fits = top[0] - base[n][0] <= kMost && top[1] - base[n][1] <= kMost;
        if (__any_sync(0xffffffffu, !fits)) {
          float f[2];
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            top[j] = fmaxf(top[j], __shfl_xor_sync(0xffffffffu, top[j], 4));
            top[j] = fmaxf(top[j], __shfl_xor_sync(0xffffffffu, top[j], 8));
            top[j] = fmaxf(top[j], __shfl_xor_sync(0xffffffffu, top[j], 16));
            const float now = top[j] - base[n][j] > kMost ? top[j] - kSet : base[n][j];
            f[j] = exp2_fast(base[n][j] - now);
            base[n][j] = now;
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
        for (int m = 0; m < 2; ++m)
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            float p = exp2_fast(fmaf(s[n][m][j], unscale[n][j & 1], -base[n][j & 1]));
            if constexpr (EDGE) p = (hidden[n] >> (4 * m + j)) & 1u ? 0.f : p;   // -inf times a scale of 0 is no number
            s[n][m][j] = p;
            sum[n][j & 1] += p;
          }
      }

      // o += V^T (p d)
#pragma unroll
      for (int k = 0; k < NB; ++k) {
        uint32_t f[4][4];   // [keys 8 i ..][features 2 g, 2 g + 1, 16 + 2 g, 17 + 2 g]
        if constexpr (Q4) {
          uint32_t x[4];
          load_matrices<true>(at + S::V_OFF + mrow + 16 * (k ^ mperm), x);
#pragma unroll
          for (int i = 0; i < 4; ++i) pairs_q4(x[i], f[i]);
        } else {
          uint32_t x[4], y[4];
          load_matrices<true>(at + S::V_OFF + mrow + 16 * ((2 * k) ^ mperm), x);
          load_matrices<true>(at + S::V_OFF + mrow + 16 * ((2 * k + 1) ^ mperm), y);
#pragma unroll
          for (int i = 0; i < 4; ++i) pairs_q8<0, 2, 1, 3>(x[i], y[i], f[i]);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          f[i][0] = add_f16x2(f[i][0], kOff0);
          f[i][1] = add_f16x2(f[i][1], kOff0);
          f[i][2] = add_f16x2(f[i][2], kOff1);
          f[i][3] = add_f16x2(f[i][3], kOff1);
        }
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          uint32_t w[4];   // of query row g, keys 2 t and 2 t + 1 of each eight
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float d = scale_of(dv[i][k / 2], k % 2);
            float w0 = s[n][i / 2][i % 2 * 2] * d, w1 = s[n][i / 2][i % 2 * 2 + 1] * d;
            if constexpr (EDGE) {   // a hidden key's scale may be anything
              w0 = (hidden[n] >> (2 * i)) & 1u ? 0.f : w0;
              w1 = (hidden[n] >> (2 * i + 1)) & 1u ? 0.f : w1;
            }
            w[i] = transpose8x8(pack_f16x2(w0, w1));
          }
#pragma unroll
          for (int m = 0; m < 2; ++m) {
            mma_f16(acc[n][2 * k], f[2 * m][0], f[2 * m][1], f[2 * m + 1][0], f[2 * m + 1][1], w[2 * m], w[2 * m + 1]);
            mma_f16(acc[n][2 * k + 1], f[2 * m][2], f[2 * m][3], f[2 * m + 1][2], f[2 * m + 1][3], w[2 * m], w[2 * m + 1]);
          }
        }
      }
    };

    int slot = 0;
    for (int tile = 0; tile < tiles; ++tile) {
      if (tile + S::STAGES - 1 < tiles) load(ring + (slot == 0 ? S::STAGES - 1 : slot - 1) * S::BYTES);
      commit();
      asm volatile("cp.async.wait_group %0;" ::"n"(S::STAGES - 1) : "memory");
      __syncwarp();
      const uint32_t at = ring + slot * S::BYTES;
      const int first = k0 + tile * kTile;
      if (first + kTile - 1 > all_to || first < all_from) step(std::true_type{}, at, first);
      else step(std::false_type{}, at, first);
      __syncwarp();   // the slot is read: the next load into it may begin
      slot = slot == S::STAGES - 1 ? 0 : slot + 1;
    }
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        sum[n][j] += __shfl_xor_sync(0xffffffffu, sum[n][j], 4);
        sum[n][j] += __shfl_xor_sync(0xffffffffu, sum[n][j], 8);
        sum[n][j] += __shfl_xor_sync(0xffffffffu, sum[n][j], 16);
      }
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int i = 0; i < 2 * NB; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[n][i][j] *= Q4 && i % 2 ? 1048576.f : 16777216.f;   // the operands' 2^-20 and 2^-24
  };

  // The sums of the last run as they are, rows of D.
  auto put = [&](float* o, float2* ml) {
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int col = n * 8 + 2 * t + j;
        if (g == 0) ml[col] = make_float2(base[n][j], sum[n][j]);
#pragma unroll
        for (int i = 0; i < 2 * NB; ++i)
          *reinterpret_cast<float2*>(o + col * D + 16 * i + 2 * g) = make_float2(acc[n][i][j], acc[n][i][j + 2]);
      }
  };
  // ... as the result of a head.
  auto finish = [&](int b, int h) {
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int r = r0 + n * 8 + 2 * t + j;
        if (r >= a.R) continue;
        const float l = sum[n][j], inv = l == 0.f ? 0.f : 1.f / l;
        __nv_bfloat16* o = a.o + q_offset(a, b, h, r) + 2 * g;
#pragma unroll
        for (int i = 0; i < 2 * NB; ++i)
          *reinterpret_cast<uint32_t*>(o + 16 * i) = tc::pack_bf16x2(acc[n][i][j] * inv, acc[n][i][j + 2] * inv);
        if (g == 0) a.lse[((size_t)b * a.Hq + h * a.G) * a.Sq + r] = l == 0.f ? 0.f : lse_of(base[n][j], l);
      }
  };

  const size_t block = (size_t)blockIdx.y * gridDim.x + blockIdx.x;
  constexpr int RING = kWarps * S::STAGES * S::BYTES, FIRST = RING > left_bytes(kWarps, D, NT) ? RING : left_bytes(kWarps, D, NT);
  float* so = reinterpret_cast<float*>(smem);   // of the heads that runs end in, once every warp is done with its ring
  float2* sml = reinterpret_cast<float2*>(smem + kWarps * ROWS * D * 4);
  float* fo = reinterpret_cast<float*>(smem + FIRST);   // of the heads that end inside a run
  float2* fml = reinterpret_cast<float2*>(smem + FIRST + kWarps * ROWS * D * 4);
  if constexpr (SLICES && left_in_memory(D, Q4, NT)) {
    fo = a.warp_o + block * kWarps * ROWS * D;
    fml = a.warp_ml + block * kWarps * ROWS;
  }
  const int rows = min(ROWS, a.R - r0);

  if constexpr (!SLICES) {   // every warp a part of the head's tiles, and then rows of their sums
    const int b = blockIdx.x / a.c.Hkv, h = blockIdx.x % a.c.Hkv;
    const Range kr = key_range(a, length_of(a, b), report && h == 0 && threadIdx.x == 0);
    const int n = (kr.len - kr.lo + kTile - 1) / kTile, first = n * warp / kWarps;
    run(b, h, kr, first, n * (warp + 1) / kWarps - first);
    asm volatile("cp.async.wait_all;" ::: "memory");
    __syncthreads();
    put(so + warp * ROWS * D, sml + warp * ROWS);
    __syncthreads();
    for (int col = warp; col < rows; col += kWarps) {
      const float2 ml = lane < kWarps ? sml[lane * ROWS + col] : make_float2(-CUDART_INF_F, 0.f);
      const float top = warp_max(ml.x), w = lane < kWarps ? exp2_fast(ml.x - top) : 0.f, l = warp_sum(w * ml.y);
      float o[D / 32];
#pragma unroll
      for (int j = 0; j < D / 32; ++j) o[j] = 0.f;
#pragma unroll 4
      for (int k = 0; k < kWarps; ++k) add_part(o, __shfl_sync(0xffffffffu, w, k), reinterpret_cast<const V*>(so + (k * ROWS + col) * D)[lane]);
      store_row<D>(a, b, h, r0 + col, o, l, top, true, nullptr, nullptr);
    }
  } else {
    if (lane < 2) left_head[2 * warp + lane] = -1;
    __syncwarp();

    bool keep = false;     // the last run is of a head that is left to the block
    make_list<kWarps * 32>(a, list, report);
    const Slices slices((unsigned)list[a.c.B] * a.c.Hkv, gridDim.x);
    const unsigned slice = slices.begin(blockIdx.x);   // the first unit of the block
    const Slices runs(slices.begin(blockIdx.x + 1) - slice, kWarps);
    unsigned at = slice + runs.begin(warp);
    const unsigned end = slice + runs.begin(warp + 1);
    while (at < end) {
      const int b = sequence_of(list, a.c.B, a.c.Hkv, at);
      const unsigned n = list[b + 1] - list[b], off = at - (unsigned)list[b] * a.c.Hkv;
      const unsigned from = off % n, to = min(n, from + (end - at));   // of the head's units
      const int h = (int)(off / n), tile = max((int)from - kStart, 0), take = (int)to - kStart - tile;
      at += to - from;
      if (take <= 0) continue;   // no more than the head's beginning
      run(b, h, key_range(a, length_of(a, b), false), tile, take);
      if (take == (int)n - kStart) {
        finish(b, h);
        continue;
      }
      keep = at == end;   // the run's last head stays in registers; its first is put away
      if (lane == 0) {
        left_head[2 * warp + keep] = b * a.c.Hkv + h;
        left_tiles[2 * warp + keep] = take;
      }
      if (!keep) put(fo + warp * ROWS * D, fml + warp * ROWS);
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
    __syncthreads();
    if (keep) put(so + warp * ROWS * D, sml + warp * ROWS);
    __syncthreads();

    // Heads that warps share, a row of one of them for each warp in turn: lane k looks after part k, which is of warp k / 2:
    // the head its run begins in, and the one it ends in. Its lanes k + SPAN, ... do so too, for sums over SPAN lanes.
    constexpr int PARTS = 2 * kWarps, SPAN = PARTS <= 8 ? 8 : PARTS <= 16 ? 16 : 32;
    constexpr uint32_t FIRST_LANES = 0xffffffffu >> (32 - SPAN);
    static_assert(PARTS <= 32, "a part a lane");
    const int my_part = lane % SPAN;
    const int my_head = my_part < PARTS ? left_head[my_part] : -1;
    const int my_tiles = lane < PARTS && my_head >= 0 ? left_tiles[lane] : 0;
    const float2* my_ml = (my_part & 1 ? sml : fml) + my_part / 2 * ROWS;
    int unit = warp;   // counts down the rows until this warp's next one
    for (uint32_t rest = __ballot_sync(0xffffffffu, my_head >= 0) & FIRST_LANES; rest != 0;) {
      const int head = __shfl_sync(0xffffffffu, my_head, __ffs(rest) - 1);
      const bool mine = my_head == head;
      const uint32_t parts = __ballot_sync(0xffffffffu, mine) & FIRST_LANES;
      rest &= ~parts;
      if (unit >= rows) {
        unit -= rows;
        continue;
      }
      const int b = head / a.c.Hkv, h = head % a.c.Hkv;
      const int n = list[b + 1] - list[b];
      const bool whole = __reduce_add_sync(0xffffffffu, mine ? my_tiles : 0) == n - kStart;
      const int part = (unsigned)list[b] * a.c.Hkv + (unsigned)h * n > slice;   // it begins inside the slice
      for (; unit < rows; unit += kWarps) {
        const int col = unit, r = r0 + col;
        const float2 ml = mine ? my_ml[col] : make_float2(-CUDART_INF_F, 0.f);
        float top = ml.x;
#pragma unroll
        for (int x = SPAN / 2; x > 0; x >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, x));
        const float w = mine ? exp2_fast(ml.x - top) : 0.f;
        float l = w * ml.y;
#pragma unroll
        for (int x = SPAN / 2; x > 0; x >>= 1) l += __shfl_xor_sync(0xffffffffu, l, x);
        float o[D / 32];
#pragma unroll
        for (int j = 0; j < D / 32; ++j) o[j] = 0.f;
#pragma unroll 1
        for (uint32_t m = parts; m != 0; m &= m - 1) {
          const int k = __ffs(m) - 1;
          const float wk = __shfl_sync(0xffffffffu, w, k);
          add_part(o, wk, reinterpret_cast<const V*>((k & 1 ? so : fo) + k / 2 * ROWS * D + col * D)[lane]);
        }
        store_row<D>(a, b, h, r, o, l, top, whole, a.part_o + (block * 2 + part) * ROWS * D + col * D,
                     a.part_ml + (block * 2 + part) * ROWS + col);
      }
      unit -= rows;
    }
  }
}

// Joins what several blocks left of one query row's head: the row's warps take the parts in turn, and are joined in
// order. A head that one block had is finished; one without keys is zeros. Where the parts are is known before they are
// there: only loads and sums are left when the kernel before has ended.
template <int D, int WARPS>
__global__ void __launch_bounds__(256) decode_join_kernel(DecodeArgs a, int blocks, int rows_per, long long all_rows) {
  constexpr int F = D / 32, AHEAD = 8;
  using V = std::conditional_t<F == 4, float4, float2>;
  __shared__ int list[kMaxListed + 1];
  __shared__ float so[8][D];
  __shared__ float2 sml[8];
  const int lane = threadIdx.x & 31, warp = (threadIdx.x >> 5) % WARPS;
  const long long row = blockIdx.x * (8LL / WARPS) + (threadIdx.x >> 5) / WARPS;
  const bool in = row < all_rows;
  const unsigned u = in ? (unsigned)row : 0u, i = u % a.Sq, head = u / a.Sq % a.Hq;
  const int b = (int)(u / a.Sq / a.Hq), h = (int)(head / a.G), r = (int)(head % a.G * a.Sq + i);   // row of the key/value head
  make_list<256>(a, list, false);
  const Slices slices((unsigned)list[a.c.B] * a.c.Hkv, blocks);
  const unsigned n = list[b + 1] - list[b], begin = (unsigned)list[b] * a.c.Hkv + (unsigned)h * n;
  int c0 = 0, c1 = -1, first_part = 0;
  if (n > 0) {
    c0 = (int)slices.of(begin + kStart);   // the first tile's, and the last one's
    c1 = (int)slices.of(begin + n - 1);
    first_part = begin > slices.begin(c0);   // of c0: the head its slice begins in, or ends in
  }
  const size_t parts = (size_t)(r / rows_per) * blocks;
  const int col = r % rows_per;
  auto place = [&](int c) { return ((parts + c) * 2 + (c == c0 ? first_part : 0)) * rows_per + col; };
  wait_for_kernel_before();
  if (!in || (n > 0 && c0 == c1)) return;
  float top = -CUDART_INF_F, l = 0.f, o[F];
#pragma unroll
  for (int j = 0; j < F; ++j) o[j] = 0.f;
  for (int c = c0 + warp; c <= c1; c += 32 * WARPS) {   // 32 parts at a time, one of them for each lane to look at
    const int count = min(32, (c1 - c) / WARPS + 1);
    float2 ml = make_float2(-CUDART_INF_F, 0.f);
    if (lane < count) ml = a.part_ml[place(c + lane * WARPS)];
    V v[AHEAD];
    auto fetch = [&](int k0) {
#pragma unroll
      for (int k = 0; k < AHEAD; ++k)
        if (k0 + k < count) v[k] = reinterpret_cast<const V*>(a.part_o + place(c + (k0 + k) * WARPS) * D)[lane];
    };
    fetch(0);
    const float now = fmaxf(top, warp_max(ml.x)), back = top == -CUDART_INF_F ? 0.f : exp2_fast(top - now);
    const float w = lane < count ? exp2_fast(ml.x - now) : 0.f;
    top = now;
    l = l * back + warp_sum(w * ml.y);
#pragma unroll
    for (int j = 0; j < F; ++j) o[j] *= back;
    for (int k0 = 0; k0 < count; k0 += AHEAD) {
      if (k0 > 0) fetch(k0);
#pragma unroll
      for (int k = 0; k < AHEAD; ++k) {
        const float wk = __shfl_sync(0xffffffffu, w, (k0 + k) & 31);
        if (k0 + k < count) add_part(o, wk, v[k]);
      }
    }
  }
  if constexpr (WARPS > 1) {
    if (lane == 0) sml[warp] = make_float2(top, l);
#pragma unroll
    for (int j = 0; j < F; ++j) so[warp][lane * F + j] = o[j];
    __syncthreads();
    if (warp != 0) return;
    const float2 ml = lane < WARPS ? sml[lane] : make_float2(-CUDART_INF_F, 0.f);
    top = warp_max(ml.x);
    const float w = ml.x == -CUDART_INF_F ? 0.f : exp2_fast(ml.x - top);   // -inf: a warp without a part
    l = warp_sum(w * ml.y);
#pragma unroll
    for (int j = 0; j < F; ++j) o[j] = 0.f;
#pragma unroll
    for (int k = 0; k < WARPS; ++k) {
      const float wk = __shfl_sync(0xffffffffu, w, k);
#pragma unroll
      for (int j = 0; j < F; ++j) o[j] = fmaf(wk, so[k][lane * F + j], o[j]);
    }
  }
  store_row<D>(a, b, h, r, o, l, top, true, nullptr, nullptr);
}

struct DecodePlan {
  int nt, row_blocks, warps;
  bool slices;
  long long blocks;
  size_t part_ml, warp_o, warp_ml, total;   // offsets in the workspace; part_o is at 0
};

DecodePlan plan_decode(const fa_decode_params* p, const CacheView& c) {
  DecodePlan d{};
  const int R = p->Hq / c.Hkv * p->Sq;
  d.nt = R <= 8 ? 1 : 2;
  d.row_blocks = (R + 8 * d.nt - 1) / (8 * d.nt);
  const long long most = p->window > 0 ? (long long)p->window + p->Sq + kTile - 1 : c.S;
  const int keys = (int)(most < c.S ? most : c.S);
  const int tiles = (keys + kTile - 1) / kTile;
  const long long heads = (long long)c.B * c.Hkv;
  // One head a block, and no second kernel, when a head is at most four tiles a warp, and when the list of sequences is too
  // long for shared memory (heads enough for every SM then). Where a block has an SM to itself it has as many warps as that
  // holds, and slices, which spread the tiles over all SMs, cost list, ends and second kernel, as much as three tiles
  // of all warps; up to six a warp, as heads may be of any length below S. 128 heads of 128 features in 4 bits with
  // 825 to 1100 keys took 11.8 us in slices and 8.2 in a block each, 32 heads 8.4 and 8.2, 32 heads of twice the length
  // 9.9 and 11.1, 128 of 8400 keys 31.2 and 30.6.
  const int sms = sm_count();
  const long long blocks = heads * d.row_blocks;
  const bool alone = blocks <= sms;
  d.warps = alone ? wide_of(c.D, d.nt) : warps_of(c.D);
  const bool few = alone ? tiles <= 6 * d.warps && tiles * (sms - blocks) <= 3LL * d.warps * sms : tiles <= 4 * d.warps;
  d.slices = !few && c.B <= kMaxListed;
  // Wide blocks for slices as well where there are heads enough that most are whole in one (64 sequences of 1024 to 8192 keys in
  // 4 bits, 32 heads on 8: 61.6 us, 62.9 in narrow ones; one sequence of 67584 keys, 16 heads on 4: 16.2 and 15.9).
  const bool wide = d.nt == 1 && heads >= 2LL * sms;
  if (d.slices) d.warps = wide ? wide_of(c.D, d.nt) : warps_of(c.D);
  const int warps = d.warps;
  d.blocks = heads;
  if (d.slices) {
    // as many blocks as the SMs hold at a time, no slice below a tile a warp
    const long long all = (long long)(wide ? 1 : held_of(c.D, d.nt)) * sms / d.row_blocks, some = heads * tiles / warps;
    d.blocks = all < some ? all : some;
    if (d.blocks < 1) d.blocks = 1;
    const size_t rows = (size_t)d.row_blocks * d.blocks * d.nt * 8;
    d.part_ml = align_up(2 * rows * c.D * 4);
    d.warp_o = d.part_ml + align_up(2 * rows * 8);
    const size_t left = left_in_memory(c.D, c.q4, d.nt) ? warps * rows : 0;
    d.warp_ml = d.warp_o + align_up(left * c.D * 4);
    d.total = d.warp_ml + align_up(left * 8);
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

template <int D, bool Q4, int NT, bool SLICES, int WARPS>
cudaError_t launch_decode(const DecodeArgs& a, dim3 grid, cudaStream_t st) {
  using S = Slot<D, Q4>;
  constexpr int ring = WARPS * S::STAGES * S::BYTES, left = left_bytes(WARPS, D, NT);
  constexpr int bytes = (ring > left ? ring : left) + (SLICES && !left_in_memory(D, Q4, NT) ? left : 0);
  auto kernel = decode_kernel<D, Q4, NT, SLICES, WARPS>;
  static std::atomic<uint64_t> allowed{0};
  const cudaError_t e = allow_shared(kernel, bytes, allowed);
  if (e != cudaSuccess) return e;
  kernel<<<grid, WARPS * 32, bytes, st>>>(a);
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
  if (plan.slices) {
    char* w = static_cast<char*>(ws);
    a.part_ml = reinterpret_cast<float2*>(w + plan.part_ml);
    a.warp_o = reinterpret_cast<float*>(w + plan.warp_o);
    a.warp_ml = reinterpret_cast<float2*>(w + plan.warp_ml);
  }
  a.status = device_status_ptr();
  a.scale2 = p->scale * 1.4426950408889634f;
  a.Hq = p->Hq;
  a.Sq = p->Sq;
  a.window = p->window;
  a.layout = p->layout;
  a.G = p->Hq / cv.Hkv;
  a.R = a.G * p->Sq;
  if (plan.row_blocks > 65535 || plan.blocks > 0x7fffffffLL || rows > 0x7fffffffULL) { set_error("too many query rows for one launch"); return FA_ERR_UNSUPPORTED; }
  const dim3 grid((unsigned)plan.blocks, (unsigned)plan.row_blocks);
  cudaStream_t cs = (cudaStream_t)stream;
  auto go = [&](auto dim, auto q4) {
    constexpr int D = decltype(dim)::value;
    constexpr bool Q4 = decltype(q4)::value;
    auto of = [&](auto nt) {
      constexpr int NT = decltype(nt)::value, W = warps_of(D), WIDE = wide_of(D, NT);
      if (plan.slices) {
        if constexpr (NT == 1)
          if (plan.warps == WIDE) return launch_decode<D, Q4, NT, true, WIDE>(a, grid, cs);
        return launch_decode<D, Q4, NT, true, W>(a, grid, cs);
      }
      return plan.warps == W ? launch_decode<D, Q4, NT, false, W>(a, grid, cs) : launch_decode<D, Q4, NT, false, WIDE>(a, grid, cs);
    };
    return plan.nt == 1 ? of(std::integral_constant<int, 1>{}) : of(std::integral_constant<int, 2>{});
  };
  using D64 = std::integral_constant<int, 64>;
  using D128 = std::integral_constant<int, 128>;
  cudaError_t e;
  if (cv.q4) e = cv.D == 64 ? go(D64{}, std::true_type{}) : go(D128{}, std::true_type{});
  else e = cv.D == 64 ? go(D64{}, std::false_type{}) : go(D128{}, std::false_type{});
  if (e == cudaSuccess && plan.slices) {
    // a warp for a row where blocks have heads enough that one is in two or three parts, else a block of eight
    const int blocks = (int)plan.blocks, per = plan.nt * 8;
    const bool few = (long long)cv.B * cv.Hkv * 4 >= plan.blocks;
    const unsigned n = (unsigned)(few ? (rows + 7) / 8 : rows);
    auto join = cv.D == 64 ? (few ? decode_join_kernel<64, 1> : decode_join_kernel<64, 8>)
                           : (few ? decode_join_kernel<128, 1> : decode_join_kernel<128, 8>);
    e = launch_after(join, dim3(n), 256, cs, a, blocks, per, (long long)rows);
    count_launches(1);
  }
  return cuda_status(e, "decode launch");
}

}  // extern "C"
