// Where a key of a paged cache lies: key j of sequence b is row j % P of page table[b, j / P] of the pool (fa_pages). What it costs:
// a token of 64 sequences of 1024 to 8192 keys in 4 bits, 32 heads on 8, is decoded in 68.3 us in pages of 64 keys and in 62.5 in one
// piece; 4 prompts of 4095 tokens, 8 heads, are written in 8 bits in 25.9 and read back in 27.1 us, in pages of 16.
#pragma once

#include <stdint.h>

#include "fa_internal.h"

namespace fa {

// Row of the pool's planes that holds key j of head h of sequence b; -1, and a report, where the table names no page of the
// pool. Keys j .. j + 15 of a j that is a multiple of 16 lie in one page, as P is one too: their rows follow each other.
// j / P is a product: with n = j / 16 and e = magic P / 16 - 2^40, both below 2^20, n magic / 2^40 is n / (P / 16) and less
// than n e / 2^40 / (P / 16) < 1 / (P / 16) more, which cannot reach the next whole number.
__device__ __forceinline__ unsigned page_index(const PageView& p, unsigned j) {
  return (unsigned)(((unsigned long long)(j >> 4) * p.magic) >> 40);
}
// ... with the table's entry for key j at hand.
__device__ __forceinline__ long long row_in_page(const PageView& p, int page, int Hkv, int h, unsigned j, unsigned* status) {
  if ((unsigned)page >= p.pages) {
    if (status != nullptr) atomicCAS(status, 0u, 0x40000000u | kSitePage);
    return -1;
  }
  return ((long long)page * Hkv + h) * p.P + (j - page_index(p, j) * p.P);
}
__device__ __forceinline__ long long page_row(const PageView& p, int Hkv, int b, int h, unsigned j, unsigned* status) {
  return row_in_page(p, __ldg(p.table + b * p.stride + page_index(p, j)), Hkv, h, j, status);
}

}  // namespace fa
