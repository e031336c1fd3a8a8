/*
 * ft_attn.h -- C ABI of the attention operators that run next to the expert
 * layer in a decode or prefill step, on GB300 (sm_103a).  Part of
 * libft_moe.so; the conventions of ft_moe.h hold (caller-owned memory, work
 * only enqueued on `stream`, host errors returned before anything is
 * enqueued, device-only errors in the caller's dev_status word).
 *
 *   ft_rope_freqs   rotary frequencies, scaled for long contexts (host)
 *   ft_rope         rotate the heads of q or k
 *   ft_rope_by_axes, ft_kv_append_by_axes
 *                   the same, and the cache write, with several positions a
 *                   token (time, height, width), one for each channel pair
 *   ft_kv_append    write new key and value rows into a paged cache, quantised
 *                   as they are written; rotates k (and q) in the same launch
 *   ft_kv_gather    read cached rows back as dense rows
 *   ft_attn_decode  attention of one new token a row over the paged cache,
 *                   split over the cache's length and joined
 *
 * A decode step: ft_kv_append (q, k, v of the new tokens), ft_attn_decode,
 * the output projection, then the expert layer.
 */
#ifndef FT_ATTN_H
#define FT_ATTN_H

#include "ft_moe.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Element types of dense tensors. */
enum { FT_DT_BF16 = 0, FT_DT_F16 = 1, FT_DT_F32 = 2 };

/*
 * Formats of a cached row (the D values of one token's key or value head).
 *   FT_KV_BF16, FT_KV_F16: the values themselves.
 *   FT_KV_E4M3: D bytes c and an exponent e: value = c * 2^e.  e is the
 *     smallest integer >= -64 with max|x| <= 448 * 2^e, c the nearest E4M3
 *     value of x * 2^-e (ties to even).  A power of two costs E4M3 no
 *     precision (its codes are themselves floating) and makes the scaling
 *     exact in both directions.
 *   FT_KV_NVFP4: D/2 bytes of E2M1 codes (low nibble = even element), D/16
 *     E4M3 block scales b, and an exponent e: value = code * b * 2^e.  e is
 *     the smallest integer >= -64 with max|x| <= 6 * 448 * 2^e; b the nearest
 *     E4M3 value of max|block| * 2^-e / 6; code the nearest E2M1 value of
 *     x * 2^-e / b (0 where b is 0).
 * Exponents are stored as one byte e + 127 a row; bytes that no row is written
 * with (e below -64, above 120, with FT_KV_NVFP4 above 117) are read as the
 * nearest that one is.  The maxima are those of the finite elements.  An
 * infinity has the largest code: with FT_KV_E4M3 448 * 2^e, with FT_KV_NVFP4
 * 6 * b * 2^e of its block, 0 where the block's finite elements are all 0.  A
 * NaN stays NaN (with NVFP4, its whole block of 16).
 */
enum { FT_KV_BF16 = 0, FT_KV_F16 = 1, FT_KV_E4M3 = 2, FT_KV_NVFP4 = 3 };

/*
 * One layer's cache.  Row (page, head, slot) has the index
 *   r = page * page_stride + head * head_stride + slot * slot_stride
 * (strides in rows, so both [page][head][slot] and [page][slot][head] orders,
 * and layers interleaved in one allocation, can be described), the same for
 * keys and values; its codes start at k + r * row bytes (ft_kv_row_bytes), its
 * exponent byte at k_scale + r, its block scales at k_block + r * (D / 16).
 * Arrays 16-byte aligned, the scale arrays allocated in whole 4-byte words
 * (they are read as words); scale and block arrays NULL where the format has
 * none.  Limits: D a multiple of 16 (FT_KV_NVFP4: of 32), at most 256; every
 * row index below 2^31 - 1.
 */
typedef struct {
  int32_t fmt;
  int32_t Hkv;
  int32_t D;
  int32_t page_size;
  int64_t n_pages;
  int64_t page_stride, head_stride, slot_stride;
  void* k;
  void* v;
  uint8_t* k_scale;
  uint8_t* v_scale;
  uint8_t* k_block;
  uint8_t* v_block;
} ft_kv_cache;

/*
 * Which pages hold a sequence: pages[s * stride + i] is the page of sequence
 * s's tokens i * page_size .. (i + 1) * page_size - 1.  Entries past a
 * sequence's length are not read.  A page outside [0, n_pages) or a sequence
 * outside [0, n_seqs) records FT_ERR_BAD_ID; the token is skipped.
 */
typedef struct {
  const int32_t* pages;
  int64_t stride;
  int32_t max_pages;
  int32_t n_seqs;
} ft_page_table;

/* Rows of heads: element (t, h, d) at base + t * token_stride + h * head_stride + d (strides in elements). */
typedef struct {
  void* base;
  int64_t token_stride, head_stride;
} ft_rows;

/*
 * Rotary positions.  Channel pair i (of rot_dim / 2) of a head turns by
 * pos * freqs[i] * 2^-64 turns: freqs is a device array of rot_dim / 2
 * fixed-point fractions of a turn, so that the product wraps modulo one turn
 * exactly and far positions lose nothing.  The pair is (x[2i], x[2i+1]) when
 * interleaved is non-zero, else (x[i], x[i + rot_dim/2]).  The rotated
 * channels are multiplied by mscale; channels rot_dim.. pass through.
 */
typedef struct {
  const int64_t* freqs;
  int32_t rot_dim;
  int32_t interleaved;
  float mscale;
} ft_rope_table;

/*
 * ft_rope_freqs -- freqs_host[i], i < rot_dim / 2, of base^(-2i/rot_dim)
 * radians a position, changed for contexts longer than the trained orig_len:
 *   FT_ROPE_PLAIN           as it is
 *   FT_ROPE_LINEAR          divided by factor
 *   FT_ROPE_BASE            base replaced by base * factor^(rot_dim / (rot_dim - 2))
 *   FT_ROPE_PARTS_BY_TURNS  f * (g + (1 - g) / factor), g rising from 0 to 1 as
 *                           the turns that f makes in orig_len go from low to high
 *   FT_ROPE_PARTS_BY_INDEX  the same with g linear in the channel index between
 *                           the (rounded outward) indices that make high and low turns
 * PLAIN reads neither factor, low, high nor orig_len; LINEAR and BASE only factor.
 */
enum {
  FT_ROPE_PLAIN = 0,
  FT_ROPE_LINEAR = 1,
  FT_ROPE_BASE = 2,
  FT_ROPE_PARTS_BY_TURNS = 3,
  FT_ROPE_PARTS_BY_INDEX = 4
};
FT_API ft_status ft_rope_freqs(int32_t rot_dim, double base, int32_t scaling, double factor, double low, double high,
                               int32_t orig_len, int64_t* freqs_host);

/*
 * ft_rope -- out[t, h] = x[t, h] rotated to position pos[t] (dtype FT_DT_BF16
 * or FT_DT_F16; computed in fp32, rounded once).  x and out may be the same
 * rows (in place) or must not overlap.  Strides multiples of 8 elements,
 * bases 16-byte aligned, D a multiple of 8 and at most 256, rot_dim even and
 * at most D.  T or heads of 0 does nothing.
 */
FT_API ft_status ft_rope(const ft_rows* x_host, int32_t T, int32_t heads, int32_t D, int32_t dtype,
                         const int32_t* pos, const ft_rope_table* rope_host, const ft_rows* out_host, void* stream);

/*
 * Several axes: a token has a position on each, and channel pair i turns by that
 * on axis[i].  Axis a's positions are pos[a * pos_stride + t], t < T (pos_stride
 * at least T, or 0: the same on every axis).  axis: a device array of rot_dim / 2 bytes; one past n_axes - 1
 * counts as n_axes - 1.
 */
enum { FT_ROPE_MAX_AXES = 8 };
typedef struct {
  const uint8_t* axis;
  int32_t n_axes;
  int64_t pos_stride;
} ft_rope_axes;

/*
 * ft_rope_sections -- axis_host[i], i < rot_dim / 2, from the number of pairs
 * that turn by each of n axes (together rot_dim / 2): one run after the other, or
 * (weave) the axes taking turns, pair i on axis i % n as long as that one has
 * pairs left, else on axis 0.  Woven sections of axes past 0 hold at most as many
 * as their turns.
 */
FT_API ft_status ft_rope_sections(int32_t rot_dim, const int32_t* sections_host, int32_t n, int32_t weave,
                                  uint8_t* axis_host);

/* ft_rope_by_axes -- ft_rope with several axes: pos [n_axes][T] as ft_rope_axes. */
FT_API ft_status ft_rope_by_axes(const ft_rows* x_host, int32_t T, int32_t heads, int32_t D, int32_t dtype,
                                 const int32_t* pos, const ft_rope_table* rope_host, const ft_rope_axes* axes_host,
                                 const ft_rows* out_host, void* stream);

/* Bytes of one cached row's codes; 0 for an unsupported (fmt, D). */
FT_API uint64_t ft_kv_row_bytes(int32_t fmt, int32_t D);

/*
 * ft_kv_append -- writes token t's k and v rows [Hkv, D] to position pos[t] of
 * sequence seq[t] (seq NULL: sequence t), for t < T; a token with pos[t] < 0
 * is not written (padding).  Two tokens must not have the same place.
 * rope_host non-NULL: k is rotated to rope_pos[t] (NULL: pos[t]) before it is
 * written, and so is q [T, Hq, D] into q_out (both NULL: no q), written for
 * padding tokens too.  Quantised keys are rounded from the rotation computed
 * to about 2^-34, so that their codes are those of the formula.  dtype (of
 * q, k, v, q_out): FT_DT_BF16 or FT_DT_F16, equal to the cache's where that is
 * 16-bit.  Alignment as ft_rope.
 */
FT_API ft_status ft_kv_append(const ft_kv_cache* cache_host, const ft_rows* k_host, const ft_rows* v_host, int32_t T,
                              int32_t dtype, const ft_page_table* table_host, const int32_t* seq, const int32_t* pos,
                              const ft_rope_table* rope_host, const int32_t* rope_pos, const ft_rows* q_host,
                              int32_t Hq, const ft_rows* q_out_host, int32_t* dev_status, void* stream);

/* ft_kv_append_by_axes -- ft_kv_append with several axes: rope_pos [n_axes][T] as ft_rope_axes, not NULL. */
FT_API ft_status ft_kv_append_by_axes(const ft_kv_cache* cache_host, const ft_rows* k_host, const ft_rows* v_host,
                                      int32_t T, int32_t dtype, const ft_page_table* table_host, const int32_t* seq,
                                      const int32_t* pos, const ft_rope_table* rope_host,
                                      const ft_rope_axes* axes_host, const int32_t* rope_pos, const ft_rows* q_host,
                                      int32_t Hq, const ft_rows* q_out_host, int32_t* dev_status, void* stream);

/*
 * ft_kv_gather -- the inverse: k_out and v_out [T, Hkv, D] (dtype bf16, f16 or
 * f32) get the values of position pos[t] of sequence seq[t]; zeros where
 * pos[t] < 0 or the page is bad.  k_out or v_out may be NULL.
 */
FT_API ft_status ft_kv_gather(const ft_kv_cache* cache_host, const ft_page_table* table_host, const int32_t* seq,
                              const int32_t* pos, int32_t T, const ft_rows* k_out_host, const ft_rows* v_out_host,
                              int32_t dtype, int32_t* dev_status, void* stream);

/*
 * ft_attn_decode -- out[t, h] = sum_j softmax_j(scale * q[t, h] . k_j) v_j over
 * the tokens j of sequence seq[t] (NULL: sequence t) with
 * max(0, lens[t] - window) <= j < lens[t] (window 0: all), key and value head
 * h / (Hq / Hkv).  lens[t] counts the new token, whose row the caller has
 * appended; it is held to max_pages * page_size.  A row that sees nothing
 * gives zeros and lse = -inf.  An infinity or NaN among the values of a 16-bit
 * cache that count gives NaN in its channel.  lse [T, Hq] fp32 (NULL: not
 * written) is the natural logarithm of sum_j exp(scale * q . k_j).
 * q: dtype bf16 or f16, equal to the cache's where that is 16-bit; out:
 * out_dtype of q's or FT_DT_F32.  Scores, statistics and sums are fp32; the
 * weights enter the value product as two 16-bit terms (bf16 for bf16 caches,
 * f16 otherwise: f16 terms end 2^36 below the heaviest weight, of 8- and 4-bit
 * rows weight times 2^value exponent).  A 16-bit output is the fp32 one rounded.
 * ws: device scratch of ft_attn_decode_workspace bytes, 256-byte aligned, of
 * any content; calls that may overlap need separate ones.
 * Limits: Hq a multiple of Hkv, T * Hq < 2^31, T <= 65535.  Work is numbered
 * in 32 bits: T * Hkv rows of max_pages * page_size tokens (of window + 15 where
 * that is less; the table's size counts, not the lengths) in tiles of 16 to 128
 * tokens, for groups of more than 32 query heads once each 32.  From 2^31 tiles
 * the call is refused with FT_ERR_UNSUPPORTED.
 */
FT_API size_t ft_attn_decode_workspace(int32_t T, int32_t Hq, int32_t Hkv, int32_t D);
FT_API ft_status ft_attn_decode(const ft_kv_cache* cache_host, const ft_rows* q_host, int32_t T, int32_t Hq,
                                int32_t dtype, const ft_page_table* table_host, const int32_t* seq,
                                const int32_t* lens, float scale, int32_t window, const ft_rows* out_host,
                                int32_t out_dtype, float* lse, void* ws, size_t ws_bytes, int32_t* dev_status,
                                void* stream);

#ifdef __cplusplus
}
#endif

#endif /* FT_ATTN_H */
