// ft_kv_index.h -- the index arithmetic of the paged key-value cache and of
// the decode attention's work split, as plain C++ that the kernels and a host
// test both compile.
#pragma once

#include <stdint.h>

#ifdef __CUDACC__
#define FT_HD __host__ __device__ __forceinline__
#else
#define FT_HD inline
#endif

namespace ft {

// Unsigned division of n < 2^31 by a fixed d in 1 .. 2^31: (n * mul) >> (31 + s)
// with mul = ceil(2^(31 + s) / d), s = ceil(log2 d), taken as the high word of
// 2 n * mul.  mul * d - 2^(31+s) < d <= 2^s, so the quotient's error
// n * (mul * d - 2^(31+s)) / (d * 2^(31+s)) stays below 1 / d and the floor is
// exact.
struct FastDiv {
  uint32_t mul;
  uint32_t shift;  // s
};

FT_HD FastDiv make_fast_div(uint32_t d) {
  uint32_t s = 0;
  while ((uint64_t(1) << s) < d) ++s;
  const uint64_t p = uint64_t(1) << (31 + s);
  return FastDiv{static_cast<uint32_t>((p + d - 1) / d), s};
}

FT_HD uint32_t fast_div(uint32_t n, FastDiv f) {
#ifdef __CUDA_ARCH__
  return __umulhi(n + n, f.mul) >> f.shift;
#else
  return static_cast<uint32_t>((static_cast<uint64_t>(n + n) * f.mul) >> 32) >> f.shift;
#endif
}

constexpr uint32_t kNoRow = 0xffffffffu;

// The cache's row numbering, as the kernels take it: every row index is below
// 2^31 - 1 (checked by the entry points), so rows and strides fit 32 bits.
struct KvIndex {
  uint32_t page_size;
  FastDiv by_page;
  uint32_t n_pages;
  uint32_t page_stride, head_stride, slot_stride;
};

// Row of head 0 of a token at `slot` of `page`; kNoRow for a page outside the cache.
FT_HD uint32_t kv_row(const KvIndex& x, int32_t page, uint32_t slot) {
  if (static_cast<uint32_t>(page) >= x.n_pages) return kNoRow;
  return static_cast<uint32_t>(page) * x.page_stride + slot * x.slot_stride;
}

// ---- the split of ft_attn_decode -------------------------------------------
// A row's tokens first..len-1 are cut into tiles of `tile` tokens from the
// multiple of 16 at or below `first`.  All (row, head block) units are numbered
// row by row, head block by head block, in one line: `lead` numbers that stand
// for what a unit costs beside its tiles, then one for each tile.  Worker c of
// n takes the numbers [c * share, (c + 1) * share).
struct RowSpan {
  int32_t begin;  // the first tile's first token (a multiple of 16)
  int32_t first;  // the first token that counts
  int32_t len;    // one past the last
  int32_t tiles;
};

// Of tiles of 2^log2 tokens.
FT_HD RowSpan row_span_log2(int32_t len, int32_t window, int32_t most, int32_t log2) {
  RowSpan r;
  if (len > most) len = most;
  if (len < 0) len = 0;
  r.len = len;
  r.first = (window > 0 && len > window) ? len - window : 0;
  r.begin = r.first & ~15;
  r.tiles = (len - r.begin + (1 << log2) - 1) >> log2;
  return r;
}

// The same of tiles of `tile` tokens, a power of two.
FT_HD RowSpan row_span(int32_t len, int32_t window, int32_t most, int32_t tile) {
  int32_t log2 = 0;
  while ((1 << log2) < tile) ++log2;
  return row_span_log2(len, window, most, log2);
}

FT_HD int32_t split_share(int32_t total, int32_t workers) { return total > workers ? (total + workers - 1) / workers : 1; }

// Numbers of a row of so many tiles and units.
FT_HD int32_t row_numbers(int32_t tiles, int32_t lead, int32_t units) { return tiles > 0 ? (tiles + lead) * units : 0; }

// What a share that has `left` numbers, the next at place `at` of a row's line,
// holds of the unit there.
struct UnitPart {
  int32_t unit;
  int32_t used;          // numbers of the share that go to it
  int32_t tile0, tiles;  // its tiles in the share (none where the share holds of its lead alone)
  int32_t rest;          // its tiles past the share
};

FT_HD UnitPart unit_part(int32_t at, int32_t left, int32_t tiles, int32_t lead) {
  UnitPart p;
  const int32_t n = tiles + lead;
  p.unit = at / n;
  const int32_t from = at - p.unit * n;
  p.used = n - from < left ? n - from : left;
  p.tile0 = from > lead ? from - lead : 0;
  const int32_t end = from + p.used - lead;  // one past its last tile in the share
  p.tiles = end > p.tile0 ? end - p.tile0 : 0;
  p.rest = tiles - (end > 0 ? end : 0);
  return p;
}

}  // namespace ft
