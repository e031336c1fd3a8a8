/*
 * ft_fp4.h -- C ABI of microscaled 4-bit matrices on GB300 (sm_103a): rows
 * quantised, read back, and multiplied with one another.  Part of
 * libft_moe.so; the conventions of ft_moe.h hold (caller-owned memory, work
 * only enqueued on `stream`, host errors returned before anything is
 * enqueued, device-only errors in the caller's dev_status word).
 *
 *   ft_fp4_quantize  rows of 16- or 32-bit values as 4-bit codes and scales
 *   ft_fp4_values    what such a matrix stands for, as dense rows
 *   ft_fp4_matmul    out = X W^T (+ add) of two 4-bit matrices, on the 4-bit
 *                    tensor cores
 *
 * A decoder block's dense projections: the weights are quantised once, the
 * activations in front of each product.  In the order FT_FP4_ROWS, quantised
 * rows are those of the expert blocks of ft_moe.h.
 */
#ifndef FT_FP4_H
#define FT_FP4_H

#include "ft_attn.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * Formats.  A value is E2M1 (0, 0.5, 1, 1.5, 2, 3, 4, 6 and their negatives)
 * times the scale of its block of consecutive values of the row.
 *   FT_FP4_NVFP4: blocks of 16 with an E4M3 scale b, and a scale s (fp32) of
 *     the row or of the matrix: value = code * b * s.
 *   FT_FP4_MXFP4: blocks of 32 with a power of two (E8M0: byte e + 127).
 */
enum { FT_FP4_NVFP4 = 0, FT_FP4_MXFP4 = 1 };

/*
 * Orders of the block scales, of rows of n = K / block of them.
 *   FT_FP4_TILES: tiles of 128 rows x 4 scales, 512 bytes each, those of the
 *     same rows one after the other; in a tile, the four scales of row r are
 *     the bytes (r % 32) * 16 + (r / 32) * 4 ...  This is what the tensor cores
 *     take, and what ft_fp4_matmul needs.  Bytes for rows past the last are
 *     neither written nor used; those for scales past a row's last are written
 *     as 0 and must not be NaN (0x7f, 0xff) where a product reads them.
 *   FT_FP4_ROWS: [rows][n].
 */
enum { FT_FP4_TILES = 0, FT_FP4_ROWS = 1 };

/*
 * A matrix [rows, K].  codes: row r's K / 2 bytes (low nibble = even element)
 * at codes + r * pitch; codes and pitch 16-byte aligned.  scales: of
 * ft_fp4_scale_bytes, 16-byte aligned.  scale (NVFP4; MXFP4: NULL): row r's at
 * scale + r * scale_stride, so that stride 0 is one scale of the whole matrix;
 * NULL stands for 1.  K is a positive multiple of the block, rows below 2^31.
 */
typedef struct {
  int32_t fmt;
  int32_t order;
  int64_t rows;
  int64_t K;
  int64_t pitch;
  uint8_t* codes;
  uint8_t* scales;
  float* scale;
  int64_t scale_stride;
} ft_fp4_matrix;

/* Bytes of a matrix's block scales; 0 for an unsupported (fmt, order, rows, K). */
FT_API uint64_t ft_fp4_scale_bytes(int32_t fmt, int32_t order, int64_t rows, int64_t K);

/*
 * ft_fp4_quantize -- rows x [rows, K] (dtype bf16, f16 or f32, row r at
 * r * stride elements) into the matrix.
 *   NVFP4, given = 0: s = 2^e of each row is written to scale (scale_stride 1),
 *     e the smallest integer >= -64 with max|x| <= 6 * 448 * 2^e; z = x / s.
 *   NVFP4, given != 0: s is read from scale; z = fl(x * fl(1 / s)) in fp32.
 *     b = the nearest E4M3 value of max|z of the block| / 6, at most 448; code =
 *     the nearest E2M1 value of z / b, 0 where b is 0.
 *   MXFP4: the block's scale is 2^e, e = floor(log2 max|x|) - 2 held to
 *     -127 .. 127 (-127 for zeros); code = the nearest E2M1 value of x / 2^e.
 * Codes past 6 are 6; ties go to the even code; all of it as in exact
 * arithmetic.  The maxima are those of finite values.  An infinity has the
 * largest code of its sign (0 where b is 0); a NaN makes its block's scale NaN.
 * Strides multiples of 8 elements (f32: 4), x 16-byte aligned.  Rows of 0 do
 * nothing.
 */
FT_API ft_status ft_fp4_quantize(const void* x, int64_t stride, int32_t dtype, const ft_fp4_matrix* m_host,
                                 int32_t given, void* stream);

/*
 * ft_fp4_values -- out [rows, K] (dtype bf16, f16 or f32, row r at r * stride
 * elements) = the matrix's values: fl(code * b * s) in fp32, rounded to the
 * output's type.  Strides and alignment as ft_fp4_quantize; rows of out must not
 * overlap.
 */
FT_API ft_status ft_fp4_values(const ft_fp4_matrix* m_host, void* out, int64_t stride, int32_t dtype, void* stream);

/*
 * ft_fp4_matmul -- out[t, n] = sum_k X[t, k] W[n, k] (+ add[t, n]) for X
 * [T, K] and W [N, K] of the same format, both in the order FT_FP4_TILES.  out
 * and add [T, N] (dtype bf16, f16 or f32; rows at stride elements, any
 * alignment of the type); add NULL: nothing is added; add may be out itself, or
 * one row for all tokens (stride 0).  Rows of out must not overlap.
 * Sums are fp32, of exact products of codes and block scales; each sum is
 * multiplied by the two row scales, with no infinity or lost bits between the two
 * where the result has none, add is added, and the result rounded once.
 * The result of a call depends on its sizes and values alone: sums over slices
 * of K are joined in one order.
 * dev_status records FT_ERR_TIMEOUT where a bounded wait gave up; a call that
 * finds it there writes nothing.
 * Limits: T and N at most 2^31 - 1024, and fewer than 2^31 tiles (of 128 or 256
 * rows of W by 16 to 256 of X).
 */
FT_API ft_status ft_fp4_matmul(const ft_fp4_matrix* x_host, const ft_fp4_matrix* w_host, void* out, int64_t out_stride,
                               int32_t dtype, const void* add, int64_t add_stride, int32_t* dev_status, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* FT_FP4_H */
