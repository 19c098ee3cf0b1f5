// Argument checks shared by the entry points of the C ABI.
#pragma once

#include <stddef.h>
#include <stdint.h>

#include "fa_internal.h"
#include "fa_train.h"

namespace fa {

// The calling thread's fa_last_error() text.
void set_error(const char* fmt, ...);
void clear_error();

constexpr size_t kAlign = 256;
inline size_t align_up(size_t x) { return (x + kAlign - 1) / kAlign * kAlign; }

constexpr int kMaxSeq = 1 << 24;
// Largest element count of one tensor (2^40: terabytes, more than a GB300 holds). Keeps every byte
// count of the validation and every 64-bit offset in the kernels far from overflow.
constexpr double kMaxElems = 1099511627776.0;
inline bool too_large(double a, double b, double c, double d) { return a * b * c * d > kMaxElems; }

struct Span { const void* p; size_t n; const char* name; };

bool overlaps(const Span& a, const Span& b);
// Every buffer is there and 16-byte aligned; no output overlaps an input or another output (of the first two outputs the
// caller may know it: `apart`).
fa_status check_buffers(const Span* in, int nin, const Span* out, int nout, bool apart = false);
// The workspace is large enough, 256-byte aligned and overlaps none of the call's buffers.
fa_status check_ws(void* ws, size_t ws_bytes, size_t need, const Span* bufs, int n);
fa_status cuda_status(cudaError_t e, const char* what);

// An fa_view of B x S rows of H heads of D features of es bytes: fills `out` with the bytes it
// spans. `written`: its rows must not overlap. A view without rows spans nothing and may be NULL.
fa_status check_view(const fa_view* v, int B, int S, int H, int D, size_t es, bool written, const char* name, Span& out);
// Two views of which no rows overlap, although the bytes they span may: parts of one tensor that lie side by side in each
// token of it, as those of a fused projection's output do (tokens of a sequence after one another or of all sequences), or
// in turn head by head. Both have passed check_view.
bool side_by_side(const fa_view* a, int Ha, const fa_view* b, int Hb, int B, int S, int D, size_t es);
inline RowView row_view(const fa_view* v) {
  return v == nullptr ? RowView{nullptr, 0, 0, 0} : RowView{v->ptr, v->stride_b, v->stride_s, v->stride_h};
}

// Checks an fa_cache and fills `out`; the byte ranges of its four planes.
fa_status check_cache(const fa_cache* c, CacheView& out);
void cache_spans(const CacheView& c, Span out[4]);

}  // namespace fa
