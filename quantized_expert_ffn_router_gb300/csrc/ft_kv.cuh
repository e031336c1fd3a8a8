// ft_kv.cuh -- the paged key-value cache on the device: the view that the
// kernels take, host checks of the public descriptors, and the 8- and 4-bit
// conversions of cached rows.
#pragma once

#include "ft_async.cuh"
#include "ft_attn.h"
#include "ft_common.cuh"
#include "ft_dequant.cuh"
#include "ft_kv_index.h"

namespace ft {

// The greatest power-of-two scale that fp32 rows need (448 * 2^119, 6 * 448 *
// 2^116 < 2^128); kMinExponent is the least, by definition.  Exponent bytes
// outside, which no row is written with, are read as the nearer of the two.
constexpr int max_exponent(int fmt) { return fmt == FT_KV_NVFP4 ? 117 : 120; }

template <int FMT>
__device__ __forceinline__ uint32_t held_exponent(uint32_t byte) {
  return min(max(byte, 127u + kMinExponent), 127u + max_exponent(FMT));
}

// Cache and page table as kernel arguments.
struct KvView {
  uint8_t* data[2];   // keys, values
  uint8_t* scale[2];  // exponent bytes, one a row
  uint8_t* block[2];  // E4M3 block scales, D / 16 a row
  KvIndex at;
  const int32_t* pages;
  int64_t table_stride;
  uint32_t max_pages, n_seqs;
  const int32_t* seq;  // NULL: row t reads sequence t
  int32_t row_bytes;
  int32_t D, Hkv;
};

__device__ __forceinline__ int32_t kv_seq(const KvView& v, uint32_t t) { return v.seq ? v.seq[t] : static_cast<int32_t>(t); }

// Row of head 0 of position pos >= 0 of sequence s; kNoRow (and FT_ERR_BAD_ID
// recorded) for a sequence, position or page outside the table and the cache.
__device__ __forceinline__ uint32_t kv_token_row(const KvView& v, int32_t s, uint32_t pos, int32_t* status) {
  const uint32_t p = fast_div(pos, v.at.by_page);
  uint32_t row = kNoRow;
  if (static_cast<uint32_t>(s) < v.n_seqs && p < v.max_pages)
    row = kv_row(v.at, v.pages[s * v.table_stride + p], pos - p * v.at.page_size);
  if (row == kNoRow) record_status(status, FT_ERR_BAD_ID);
  return row;
}

// Host: bytes of one row's codes (0: unsupported), and the checks that turn
// the public descriptors into a view.
uint64_t kv_row_bytes(int32_t fmt, int32_t D);
ft_status kv_view(const char* what, const ft_kv_cache* c, const ft_page_table* p, const int32_t* seq, int32_t T,
                  KvView* out);
// Strides multiples of `grain` elements, base 16-byte aligned.
ft_status check_rows(const char* what, const char* name, const ft_rows* r, int64_t grain);

}  // namespace ft
