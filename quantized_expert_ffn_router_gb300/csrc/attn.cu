// attn.cu -- attention of one new token a row over the paged key-value cache.
//
// For each row t and query head h:  x_j = scale q.k_j,  o = sum_j e^(x_j - m) v_j / sum_j e^(x_j - m)
// over the row's tokens j, in one pass with a running maximum m.  Every cached
// byte is read once and used by the G = Hq / Hkv query heads of its key head:
// 4 G flops a byte pair, far below the tensor cores' ridge, so the kernel is
// bound by HBM and everything is arranged around loads in flight.
//
// Layout of the work in a warp.  Keys go straight from global memory into the
// A operand of mma.m16n8k16 (16 tokens x 16 channels, S^T = K Q^T) and values
// into the A operand of the second product (16 channels x 16 tokens,
// O^T = V^T P^T), without passing through shared memory: the order of the
// contracted index is free as long as both operands agree, so each lane loads
// 16 contiguous bytes of a row and its elements are dealt to the fragments'
// places by renaming registers (keys) or by one byte permute a register
// (values, whose contracted index runs over tokens).  With tokens and channels
// on the 16-row side, 8 query heads fill the 8-column side: no row of the
// instruction is wasted at G = 8.  P^T changes from accumulator to operand
// layout by movmatrix.  mma.sync and not tcgen05: operands that arrive in
// registers need no staging, no barrier and no TMEM round trip, and the
// tensor work is a small part of the time (each warp has 30 mma per 8 KB).
//
// 8- and 4-bit rows: a key's power-of-two scale multiplies its score; a
// value's enters the running maximum, so that the weight that is rounded to
// f16 is p_j = 2^(x_j + ev_j - m) <= 1 whatever the scales are, and the sum
// of the softmax takes p_j 2^-ev_j in fp32.
//
// Split.  The tiles of all rows and key heads are numbered in one line and cut
// into equal shares, one a CTA (lengths are read on the device, so a captured
// graph serves any lengths).  A unit (row, head block) inside one share is
// written directly; one that crosses shares leaves partial sums that
// join_kernel adds in order.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <math.h>

#include <atomic>

#include "ft_async.cuh"
#include "ft_kv.cuh"

namespace ft {
namespace {

constexpr int kWarps = 4;
constexpr int kMaxWorkers = 1024;  // CTAs of one call (sizes the workspace)
constexpr uint32_t kAll = 0xffffffffu;

struct AttnArgs {
  KvView kv;
  const uint16_t* q;
  int64_t q_tok, q_head;
  void* out;
  int64_t out_tok, out_head;
  float* lse;
  const int32_t* lens;
  float* part_o;   // [worker][2][heads of a block][D padded]
  float2* part_ml;  // [worker][2][heads of a block] (maximum, sum)
  float scale_log2;
  int32_t window, T, Hq, G;
  int32_t units;         // head blocks of a row: Hkv * blocks
  int32_t blocks;        // head blocks of a key head
  int32_t warps_h_log2;  // warps of a CTA over head tiles; the others over tokens
  int32_t block_heads;   // heads of a block
  int32_t tile;          // tokens of a CTA's tile
  int32_t most;          // max_pages * page_size
  int32_t q_f16, out_dtype, two_terms;
  int32_t workers;
  int32_t* status;
};

// --------------------------------------------------------------- warp helpers ---
template <bool F16>
__device__ __forceinline__ void mma(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                    uint32_t b1) {
  if (F16)
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t transpose8x8(uint32_t a) {
  uint32_t d;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
  return d;
}

__device__ __forceinline__ float exp2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}

template <bool F16>
__device__ __forceinline__ uint32_t pack16(float lo, float hi) {
  uint32_t d;
  if (F16)
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
  else
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
  return d;
}

template <bool F16>
__device__ __forceinline__ float2 unpack16(uint32_t w) {
  if (F16) return __half22float2(*reinterpret_cast<const __half2*>(&w));
  return make_float2(bf16_lo(w), bf16_hi(w));
}

// N words (1, 2 or 4) of a cached row: read once, kept out of L1.
template <int N>
__device__ __forceinline__ void load_row(const uint8_t* p, uint32_t (&w)[N]) {
  if constexpr (N == 4)
    asm("ld.global.nc.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]) : "l"(p));
  else if constexpr (N == 2)
    asm("ld.global.nc.v2.u32 {%0,%1}, [%2];" : "=r"(w[0]), "=r"(w[1]) : "l"(p));
  else
    asm("ld.global.nc.u32 %0, [%1];" : "=r"(w[0]) : "l"(p));
}

// How a format's rows are dealt to lanes, for heads padded to DP channels.
// Keys: piece p of a row gives lane quarter q the EK channels p*4*EK + q*EK..;
// values: piece p gives lane group g the EV channels p*8*EV + g*EV...
template <int FMT, int DP>
struct Deal {
  static constexpr bool kQuant = FMT == FT_KV_E4M3 || FMT == FT_KV_NVFP4;
  static constexpr bool kBlocks = FMT == FT_KV_NVFP4;
  static constexpr bool kF16 = FMT != FT_KV_BF16;  // operand type of the products
  static constexpr int EK = !kQuant ? 8 : !kBlocks ? 16 : DP % 128 == 0 ? 32 : 16;
  static constexpr int EV = !kQuant ? 8 : !kBlocks ? (DP % 128 == 0 ? 16 : 8) : DP % 256 == 0 ? 32 : DP % 128 == 0 ? 16 : 8;
  static constexpr int NK = DP / (4 * EK), NV = DP / (8 * EV);
  static constexpr int per = !kQuant ? 2 : kBlocks ? 8 : 4;  // elements of a word
  static constexpr int WK = EK / per, WV = EV / per;         // words of a piece
  static constexpr int row_bits = !kQuant ? 16 : kBlocks ? 4 : 8;
  // 16-token tiles that a warp has in flight at once: about 4 KB of keys
  static constexpr int kKeyBytes = 16 * DP * row_bits / 8;
  static constexpr int U = kKeyBytes >= 4096 ? 1 : kKeyBytes >= 2048 ? 2 : 4;
};

template <int FMT, int DP, int NT>
struct Warp {
  using X = Deal<FMT, DP>;
  static constexpr int U = X::U;
  static constexpr int R = (16 * U + 31) / 32;  // tokens of a step held by a lane
  static constexpr int MT = DP / 16;

  // ---- a step's rows: lane i holds those of tokens base + i (+ 32)
  __device__ static __forceinline__ void pages_of(const AttnArgs& a, const int32_t* table, int base, int first, int end,
                                                  int lane, int32_t (&page)[R]) {
#pragma unroll
    for (int i = 0; i < R; ++i) {
      const int tok = base + lane + 32 * i;
      page[i] = -1;
      if ((U > 1 || lane < 16) && tok >= first && tok < end) page[i] = table[fast_div(tok, a.kv.at.by_page)];
    }
  }
  __device__ static __forceinline__ void rows_of(const AttnArgs& a, uint32_t head_row, int base, int first, int end,
                                                 int lane, const int32_t (&page)[R], uint32_t (&row)[R]) {
#pragma unroll
    for (int i = 0; i < R; ++i) {
      const int tok = base + lane + 32 * i;
      row[i] = kNoRow;
      if ((U > 1 || lane < 16) && tok >= first && tok < end) {
        row[i] = kv_row(a.kv.at, page[i], tok - fast_div(tok, a.kv.at.by_page) * a.kv.at.page_size);
        if (row[i] == kNoRow)
          record_status(a.status, FT_ERR_BAD_ID);
        else
          row[i] += head_row;
      }
    }
  }

  // ---- keys and values of a step
  uint32_t k[U][2][X::NK][X::WK];
  uint32_t kb[X::kBlocks ? U : 1][2][X::NK];
  uint32_t v[U][4][X::NV][X::WV];
  uint32_t vb[X::kBlocks ? U : 1][4][X::NV];
  uint32_t sc[R];    // the lane's tokens' scale bytes: key | value << 8
  uint32_t valid;    // bit 2u + r: token 16u + g + 8r counts

  __device__ __forceinline__ void load_keys(const AttnArgs& a, const uint32_t (&row)[R], int g, int q) {
    valid = 0;
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const uint32_t n = __shfl_sync(kAll, row[u >> 1], ((16 * u) & 31) + g + 8 * r);
        const bool ok = n != kNoRow;
        if (ok) valid |= 1u << (2 * u + r);
        const uint8_t* src = a.kv.data[0] + static_cast<uint64_t>(n) * a.kv.row_bytes;
#pragma unroll
        for (int p = 0; p < X::NK; ++p) {
          const int d = p * 4 * X::EK + q * X::EK;
#pragma unroll
          for (int w = 0; w < X::WK; ++w) k[u][r][p][w] = 0;
          if (X::kBlocks) kb[u][r][p] = 0;
          if (ok && (p * 4 * X::EK + 4 * X::EK <= DP - 64 || d < a.kv.D)) {
            load_row(src + d * X::row_bits / 8, k[u][r][p]);
            if constexpr (X::kBlocks) {
              const uint8_t* bp = a.kv.block[0] + static_cast<uint64_t>(n) * (a.kv.D >> 4) + (d >> 4);
              kb[u][r][p] = X::EK == 32 ? *reinterpret_cast<const uint16_t*>(bp) : *bp;
            }
          }
        }
      }
    if constexpr (X::kQuant) {
#pragma unroll
      for (int i = 0; i < R; ++i) {
        sc[i] = 0x7f7f;
        if (row[i] != kNoRow) sc[i] = a.kv.scale[0][row[i]] | (a.kv.scale[1][row[i]] << 8);
      }
    }
  }

  __device__ __forceinline__ void load_values(const AttnArgs& a, const uint32_t (&row)[R], int g, int q) {
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const uint32_t n = __shfl_sync(kAll, row[u >> 1], ((16 * u) & 31) + 2 * q + (r & 1) + 8 * (r >> 1));
        const bool ok = n != kNoRow;
        const uint8_t* src = a.kv.data[1] + static_cast<uint64_t>(n) * a.kv.row_bytes;
#pragma unroll
        for (int p = 0; p < X::NV; ++p) {
          const int d = p * 8 * X::EV + g * X::EV;
#pragma unroll
          for (int w = 0; w < X::WV; ++w) v[u][r][p][w] = 0;
          if (X::kBlocks) vb[u][r][p] = 0;
          if (ok && (p * 8 * X::EV + 8 * X::EV <= DP - 64 || d < a.kv.D)) {
            load_row(src + d * X::row_bits / 8, v[u][r][p]);
            if constexpr (X::kBlocks) {
              const uint8_t* bp = a.kv.block[1] + static_cast<uint64_t>(n) * (a.kv.D >> 4) + (d >> 4);
              vb[u][r][p] = X::EV == 32 ? *reinterpret_cast<const uint16_t*>(bp) : *bp;
            }
          }
        }
      }
  }

  // s[u][nt] = S^T of tile u: (token g | g + 8) x (head 2q | 2q + 1)
  __device__ __forceinline__ void scores(const uint32_t (&qb)[MT][NT][2], float (&s)[U][NT][4]) {
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i) s[u][n][i] = 0.f;
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int p = 0; p < X::NK; ++p) {
        uint32_t f[2][X::EK / 2];  // 16-bit pairs of rows g and g + 8
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          if constexpr (!X::kQuant) {
#pragma unroll
            for (int w = 0; w < X::WK; ++w) f[r][w] = k[u][r][p][w];
          } else if constexpr (!X::kBlocks) {
#pragma unroll
            for (int w = 0; w < X::WK; ++w) {
              f[r][2 * w] = cvt_e4m3x2(k[u][r][p][w]);
              f[r][2 * w + 1] = cvt_e4m3x2(k[u][r][p][w] >> 16);
            }
          } else {
            const uint32_t b2 = cvt_e4m3x2(kb[u][r][p]);  // the block scales (one or two)
#pragma unroll
            for (int w = 0; w < X::WK; ++w) {
              uint32_t h[4];
              e2m1x8(k[u][r][p][w], h);
              const uint32_t b = __byte_perm(b2, 0, w < 2 ? 0x1010 : 0x3232);
#pragma unroll
              for (int i = 0; i < 4; ++i) f[r][4 * w + i] = mul_f16x2(h[i], b);
            }
          }
        }
#pragma unroll
        for (int i = 0; i < X::EK / 4; ++i)
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            const int st = p * (X::EK / 4) + i;
            mma<X::kF16>(s[u][n], f[0][2 * i], f[1][2 * i], f[0][2 * i + 1], f[1][2 * i + 1], qb[st][n][0], qb[st][n][1]);
          }
      }
  }

  // acc += V^T P^T of tile u; hi and lo: P^T as operand (tokens 0..7, 8..15)
  __device__ __forceinline__ void add_values(int u, const uint32_t (&hi)[NT][2], const uint32_t (&lo)[NT][2], bool two,
                                             float (&acc)[MT][NT][4]) {
    const auto step = [&](int mt, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3) {
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        mma<X::kF16>(acc[mt][n], a0, a1, a2, a3, hi[n][0], hi[n][1]);
        if (two) mma<X::kF16>(acc[mt][n], a0, a1, a2, a3, lo[n][0], lo[n][1]);
      }
    };
#pragma unroll
    for (int p = 0; p < X::NV; ++p) {
      const int m0 = p * (X::EV / 2);
#pragma unroll
      for (int w = 0; w < X::WV; ++w) {
        const uint32_t t0 = v[u][0][p][w], t1 = v[u][1][p][w], t2 = v[u][2][p][w], t3 = v[u][3][p][w];
        if constexpr (!X::kQuant) {
          step(m0 + w, __byte_perm(t0, t1, 0x5410), __byte_perm(t0, t1, 0x7632), __byte_perm(t2, t3, 0x5410),
               __byte_perm(t2, t3, 0x7632));
        } else if constexpr (!X::kBlocks) {
          // bytes of two tokens side by side, then two conversions a word
          const uint32_t x0 = __byte_perm(t0, t1, 0x5140), x1 = __byte_perm(t0, t1, 0x7362);
          const uint32_t y0 = __byte_perm(t2, t3, 0x5140), y1 = __byte_perm(t2, t3, 0x7362);
          step(m0 + 2 * w, cvt_e4m3x2(x0), cvt_e4m3x2(x0 >> 16), cvt_e4m3x2(y0), cvt_e4m3x2(y0 >> 16));
          step(m0 + 2 * w + 1, cvt_e4m3x2(x1), cvt_e4m3x2(x1 >> 16), cvt_e4m3x2(y1), cvt_e4m3x2(y1 >> 16));
        } else {
          // nibbles of two tokens side by side: even elements, odd elements
          const uint32_t m = 0x0f0f0f0fu;
          uint32_t e0[4], o0[4], e1[4], o1[4];
          e2m1x8((t0 & m) | ((t1 & m) << 4), e0);
          e2m1x8(((t0 >> 4) & m) | (t1 & ~m), o0);
          e2m1x8((t2 & m) | ((t3 & m) << 4), e1);
          e2m1x8(((t2 >> 4) & m) | (t3 & ~m), o1);
          const int sh = (X::EV == 32 && w >= 2) ? 8 : 0;
          const uint32_t b0 = cvt_e4m3x2(((vb[u][0][p] >> sh) & 0xffu) | (((vb[u][1][p] >> sh) & 0xffu) << 8));
          const uint32_t b1 = cvt_e4m3x2(((vb[u][2][p] >> sh) & 0xffu) | (((vb[u][3][p] >> sh) & 0xffu) << 8));
#pragma unroll
          for (int i = 0; i < 4; ++i)
            step(m0 + 4 * w + i, mul_f16x2(e0[i], b0), mul_f16x2(o0[i], b0), mul_f16x2(e1[i], b1), mul_f16x2(o1[i], b1));
        }
      }
    }
  }
};

// Tiles of row t; the line's length over all rows, by one warp.
__device__ __forceinline__ RowSpan span_of(const AttnArgs& a, int t) {
  return row_span(a.lens[t], a.window, a.most, a.tile);
}

__device__ __forceinline__ int64_t warp_sum64(int64_t v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(kAll, v, o);
  return v;
}

__device__ __forceinline__ int64_t tiles_before(const AttnArgs& a, int rows, int lane) {
  int64_t n = 0;
  for (int t = lane; t < rows; t += 32) n += span_of(a, t).tiles;
  return warp_sum64(n);
}

template <int DT>
__device__ __forceinline__ void store2(void* out, int64_t at, float x, float y) {
  if (DT == FT_DT_F32)
    *reinterpret_cast<float2*>(static_cast<float*>(out) + at) = make_float2(x, y);
  else
    *reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(out) + at) = pack16<DT == FT_DT_F16>(x, y);
}

__device__ __forceinline__ void store_out(const AttnArgs& a, int t, int h, int d, float x, float y) {
  const int64_t at = static_cast<int64_t>(t) * a.out_tok + static_cast<int64_t>(h) * a.out_head + d;
  if (a.out_dtype == FT_DT_F32)
    store2<FT_DT_F32>(a.out, at, x, y);
  else if (a.out_dtype == FT_DT_F16)
    store2<FT_DT_F16>(a.out, at, x, y);
  else
    store2<FT_DT_BF16>(a.out, at, x, y);
}

__device__ __forceinline__ void store_lse(const AttnArgs& a, int t, int h, float m, float l) {
  if (a.lse) a.lse[static_cast<int64_t>(t) * a.Hq + h] = l > 0.f || l != l ? (m + log2f(l)) * 0.69314718055994531f : -INFINITY;
}

// 2^(m - M), 0 where nothing was seen (m = -inf); M = -inf only with every m.
__device__ __forceinline__ float weight_of(float m, float M) { return m == -INFINITY ? 0.f : exp2_approx(m - M); }

// The weights are rescaled when a score exceeds the running reference by this
// much (in powers of two), not at every new maximum: 2^4 leaves p far inside f16.
constexpr float kSlack = 4.f;

template <int FMT, int DP, int NT>
__global__ void __launch_bounds__(kWarps * 32) attend_kernel(const AttnArgs a) {
  using X = Deal<FMT, DP>;
  using W = Warp<FMT, DP, NT>;
  constexpr int U = X::U, R = W::R, MT = DP / 16, H = 8 * NT, DS = DP + 8;
  __shared__ float red[kWarps][H][DS];
  __shared__ float2 red_ml[kWarps][H];
  pdl_launch_dependents();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, q = lane & 3;
  const int wh = warp & ((1 << a.warps_h_log2) - 1), wt = warp >> a.warps_h_log2;
  const int warps_t = kWarps >> a.warps_h_log2;

  // this CTA's share of the line, and the row it begins in
  const int64_t total = tiles_before(a, a.T, lane) * a.units;
  const int64_t share = split_share(total, a.workers);
  int64_t at = blockIdx.x * share;
  if (at >= total) return;
  const int64_t end = at + share < total ? at + share : total;
  int t = 0;
  int64_t row_at = 0;  // the row's first number
  for (int t0 = 0;; t0 += 32) {
    int64_t n = t0 + lane < a.T ? static_cast<int64_t>(span_of(a, t0 + lane).tiles) * a.units : 0;
    int64_t upto = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t y = __shfl_up_sync(kAll, upto, o);
      if (lane >= o) upto += y;
    }
    const uint32_t past = __ballot_sync(kAll, row_at + upto > at);
    if (past) {
      const int i = __ffs(past) - 1;
      t = t0 + i;
      row_at += __shfl_sync(kAll, upto - n, i);
      break;
    }
    row_at += __shfl_sync(kAll, upto, 31);
  }

  while (at < end) {
    RowSpan span = span_of(a, t);
    while (span.tiles == 0) span = span_of(a, ++t);
    const int unit = static_cast<int>((at - row_at) / span.tiles);
    const int tile0 = static_cast<int>(at - row_at - static_cast<int64_t>(unit) * span.tiles);
    const int tile1 = end - at < span.tiles - tile0 ? tile0 + static_cast<int>(end - at) : span.tiles;
    const int kv_head = unit / a.blocks;
    const int head0 = (unit - kv_head * a.blocks) * a.block_heads;  // of the key head's group

    const int32_t seq = kv_seq(a.kv, t);
    const bool bad_seq = static_cast<uint32_t>(seq) >= a.kv.n_seqs;
    if (bad_seq) record_status(a.status, FT_ERR_BAD_ID);
    const int32_t* table = a.kv.pages + static_cast<int64_t>(bad_seq ? 0 : seq) * a.kv.table_stride;
    const uint32_t head_row = static_cast<uint32_t>(kv_head) * a.kv.at.head_stride;
    const int first = span.first;
    const int stop = span.begin + tile1 * a.tile < span.len ? span.begin + tile1 * a.tile : span.len;
    const int tok_end = bad_seq ? 0 : stop;
    const int step = 16 * U * warps_t;
    int base = span.begin + tile0 * a.tile + wt * 16 * U;

    // the first rows' loads go out before the queries are prepared
    W w;
    int32_t page[R];
    uint32_t row[R];
    W::pages_of(a, table, base, first, tok_end, lane, page);

    // queries: B operand (head g of each tile), power-of-two scaled into f16 where the products are f16
    uint32_t qb[MT][NT][2];
    float mul[NT][2];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const int h = head0 + wh * H + n * 8 + g;
      const uint16_t* src = a.q + static_cast<int64_t>(t) * a.q_tok + static_cast<int64_t>(kv_head * a.G + h) * a.q_head;
      uint2 raw[MT];
#pragma unroll
      for (int st = 0; st < MT; ++st) {
        constexpr int S = X::EK / 4;
        const int d = (st / S) * 4 * X::EK + q * X::EK + (st % S) * 4;
        raw[st] = make_uint2(0, 0);
        if (h < a.G && d < a.kv.D) raw[st] = *reinterpret_cast<const uint2*>(src + d);
      }
      float up = 1.f, down = 1.f;
      if (X::kF16) {
        float amax = 0.f;
#pragma unroll
        for (int st = 0; st < MT; ++st) {
          const float2 x = a.q_f16 ? unpack16<true>(raw[st].x) : unpack16<false>(raw[st].x);
          const float2 y = a.q_f16 ? unpack16<true>(raw[st].y) : unpack16<false>(raw[st].y);
          amax = fmaxf(fmaxf(amax, fmaxf(fabsf(x.x), fabsf(x.y))), fmaxf(fabsf(y.x), fabsf(y.y)));
        }
        amax = fmaxf(amax, __shfl_xor_sync(kAll, amax, 1));
        amax = fmaxf(amax, __shfl_xor_sync(kAll, amax, 2));
        // the largest element to [128, 256): exact, undone in the scores' factor
        int e = 134 - static_cast<int>(__float_as_uint(amax) >> 23);
        e = amax > 0.f && amax <= 3.4028235e38f ? min(max(e, -120), 120) : 0;
        up = __uint_as_float((127 + e) << 23);
        down = __uint_as_float((127 - e) << 23);
      }
#pragma unroll
      for (int st = 0; st < MT; ++st) {
        if (X::kF16) {
          const float2 x = a.q_f16 ? unpack16<true>(raw[st].x) : unpack16<false>(raw[st].x);
          const float2 y = a.q_f16 ? unpack16<true>(raw[st].y) : unpack16<false>(raw[st].y);
          qb[st][n][0] = pack16<true>(x.x * up, x.y * up);
          qb[st][n][1] = pack16<true>(y.x * up, y.y * up);
        } else {
          qb[st][n][0] = raw[st].x;
          qb[st][n][1] = raw[st].y;
        }
      }
      mul[n][0] = a.scale_log2 * __shfl_sync(kAll, down, 8 * q);
      mul[n][1] = a.scale_log2 * __shfl_sync(kAll, down, 8 * q + 4);
    }

    float acc[MT][NT][4], m[NT][2], l[NT][2];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        m[n][i] = -INFINITY;
        l[n][i] = 0.f;
      }
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[mt][n][i] = 0.f;
    }

    W::rows_of(a, head_row, base, first, tok_end, lane, page, row);
    w.load_keys(a, row, g, q);
    w.load_values(a, row, g, q);
    W::pages_of(a, table, base + step, first, tok_end, lane, page);
    while (base < tok_end) {
      float s[U][NT][4];
      w.scores(qb, s);
      const uint32_t valid = w.valid;
      uint32_t scale_bytes[R];
#pragma unroll
      for (int i = 0; i < R; ++i) scale_bytes[i] = X::kQuant ? w.sc[i] : 0;
      base += step;
      W::rows_of(a, head_row, base, first, tok_end, lane, page, row);
      w.load_keys(a, row, g, q);  // of the next step: in flight during this one's weights and values

      // scores in powers of two, with the value's exponent; masked tokens -inf
      float iv[U][2];
      bool more = false;
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          float ks = 1.f, ev = 0.f;
          iv[u][r] = 1.f;
          if (X::kQuant) {
            const uint32_t b = __shfl_sync(kAll, scale_bytes[u >> 1], ((16 * u) & 31) + g + 8 * r);
            const uint32_t kb = max(b & 0xffu, 27u), vb = max(b >> 8, 27u);  // 2^-100: a byte that no writer stores
            ks = __uint_as_float(kb << 23);
            ev = static_cast<float>(static_cast<int>(vb) - 127);
            iv[u][r] = __uint_as_float((254u - vb) << 23);
          }
          const bool ok = (valid >> (2 * u + r)) & 1;
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              float& x = s[u][n][2 * r + i];
              x = X::kQuant ? fmaf(x * ks, mul[n][i], ev) : x * mul[n][i];
              x = ok ? x : -INFINITY;
              more |= x > m[n][i] + kSlack;
            }
        }
      if (__any_sync(kAll, more)) {
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            float top = m[n][i];
#pragma unroll
            for (int u = 0; u < U; ++u) top = fmaxf(top, fmaxf(s[u][n][i], s[u][n][2 + i]));
            top = fmaxf(top, __shfl_xor_sync(kAll, top, 4));
            top = fmaxf(top, __shfl_xor_sync(kAll, top, 8));
            top = fmaxf(top, __shfl_xor_sync(kAll, top, 16));
            const float c = weight_of(m[n][i], top);
            m[n][i] = top;
            l[n][i] *= c;
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
              acc[mt][n][i] *= c;
              acc[mt][n][2 + i] *= c;
            }
          }
      }
      float ref[NT][2];
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int i = 0; i < 2; ++i) ref[n][i] = m[n][i] == -INFINITY ? 0.f : m[n][i];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        uint32_t hi[NT][2], lo[NT][2];
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            const float p0 = exp2_approx(s[u][n][2 * r] - ref[n][0]), p1 = exp2_approx(s[u][n][2 * r + 1] - ref[n][1]);
            if (X::kQuant) {
              l[n][0] = fmaf(p0, iv[u][r], l[n][0]);
              l[n][1] = fmaf(p1, iv[u][r], l[n][1]);
            } else {
              l[n][0] += p0;
              l[n][1] += p1;
            }
            const uint32_t h = pack16<X::kF16>(p0, p1);
            hi[n][r] = transpose8x8(h);
            lo[n][r] = 0;
            if (!X::kF16 || a.two_terms) {
              const float2 back = unpack16<X::kF16>(h);
              lo[n][r] = transpose8x8(pack16<X::kF16>(p0 - back.x, p1 - back.y));
            }
          }
        w.add_values(u, hi, lo, !X::kF16 || a.two_terms, acc);
      }
      w.load_values(a, row, g, q);
      W::pages_of(a, table, base + step, first, tok_end, lane, page);
    }

    // the warps' sums meet in shared memory
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        l[n][i] += __shfl_xor_sync(kAll, l[n][i], 4);
        l[n][i] += __shfl_xor_sync(kAll, l[n][i], 8);
        l[n][i] += __shfl_xor_sync(kAll, l[n][i], 16);
        if (g == 0) red_ml[warp][n * 8 + 2 * q + i] = make_float2(m[n][i], l[n][i]);
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
          const int d = (mt / (X::EV / 2)) * 8 * X::EV + g * X::EV + 2 * (mt % (X::EV / 2));
          *reinterpret_cast<float2*>(&red[warp][n * 8 + 2 * q + i][d]) = make_float2(acc[mt][n][i], acc[mt][n][2 + i]);
        }
      }
    __syncthreads();
    const bool whole = tile0 == 0 && tile1 == span.tiles;
    const int64_t slot = static_cast<int64_t>(blockIdx.x) * 2 + (tile0 == 0 ? 1 : 0);
    const int heads = a.block_heads < a.G - head0 ? a.block_heads : a.G - head0;
    for (int i = threadIdx.x; i < heads * (DP / 2); i += kWarps * 32) {
      const int h = i / (DP / 2), d = 2 * (i - h * (DP / 2));
      const int x = h / H, hh = h - x * H;  // warp column and head in it
      float M = -INFINITY;
      for (int y = 0; y < warps_t; ++y) M = fmaxf(M, red_ml[(y << a.warps_h_log2) + x][hh].x);
      float L = 0.f, o0 = 0.f, o1 = 0.f;
      for (int y = 0; y < warps_t; ++y) {
        const int wi = (y << a.warps_h_log2) + x;
        const float2 ml = red_ml[wi][hh];
        const float c = weight_of(ml.x, M);
        const float2 o = *reinterpret_cast<const float2*>(&red[wi][hh][d]);
        L += c * ml.y;
        o0 += c * o.x;
        o1 += c * o.y;
      }
      if (whole) {
        const int hq = kv_head * a.G + head0 + h;
        const float inv = L == 0.f ? 0.f : 1.f / L;
        if (d < a.kv.D) store_out(a, t, hq, d, o0 * inv, o1 * inv);
        if (d == 0) store_lse(a, t, hq, M, L);
      } else {
        *reinterpret_cast<float2*>(a.part_o + (slot * a.block_heads + h) * DP + d) = make_float2(o0, o1);
        if (d == 0) a.part_ml[slot * a.block_heads + h] = make_float2(M, L);
      }
    }
    __syncthreads();  // red is free for the next unit
    at += tile1 - tile0;
    if (tile1 == span.tiles && unit == a.units - 1) {
      row_at += static_cast<int64_t>(span.tiles) * a.units;
      ++t;
    }
  }
}

// Adds the partial sums of units that crossed shares, in the shares' order,
// and answers rows that see nothing.  One CTA a (row, query head); its warps
// take every fourth partial.
template <int DP>
__global__ void __launch_bounds__(128) join_kernel(const AttnArgs a) {
  constexpr int N = DP / 32;  // channels of a lane
  __shared__ float acc_s[4][DP];
  __shared__ float2 ml_s[4];
  const int t = blockIdx.x / a.Hq, hq = blockIdx.x - t * a.Hq;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // every CTA waits, whether it has something to add or not: work after this
  // grid must also come after attend_kernel
  pdl_wait();
  const RowSpan span = span_of(a, t);
  if (span.tiles == 0) {
    for (int d = 2 * threadIdx.x; d < a.kv.D; d += 256) store_out(a, t, hq, d, 0.f, 0.f);
    if (threadIdx.x == 0) store_lse(a, t, hq, -INFINITY, 0.f);
    return;
  }
  const int64_t before = tiles_before(a, t, lane);
  const int64_t total = tiles_before(a, a.T, lane) * a.units;
  const int64_t share = split_share(total, a.workers);
  const int kv_head = hq / a.G, hg = hq - kv_head * a.G;
  const int block = hg / a.block_heads, h = hg - block * a.block_heads;
  const int64_t from = before * a.units + static_cast<int64_t>(kv_head * a.blocks + block) * span.tiles;
  const int64_t c0 = from / share, c1 = (from + span.tiles - 1) / share;
  if (c0 == c1) return;
  float m = -INFINITY, l = 0.f, acc[N];
#pragma unroll
  for (int i = 0; i < N; ++i) acc[i] = 0.f;
  for (int64_t c = c0 + warp; c <= c1; c += 4) {
    const int64_t slot = (c * 2 + (c == c0 ? 1 : 0)) * a.block_heads + h;
    const float2 ml = a.part_ml[slot];
    float o[N];
#pragma unroll
    for (int i = 0; i < N; ++i) o[i] = a.part_o[slot * DP + lane + 32 * i];
    const float top = fmaxf(m, ml.x);
    const float x = weight_of(m, top), y = weight_of(ml.x, top);
    m = top;
    l = l * x + ml.y * y;
#pragma unroll
    for (int i = 0; i < N; ++i) acc[i] = acc[i] * x + o[i] * y;
  }
  if (lane == 0) ml_s[warp] = make_float2(m, l);
#pragma unroll
  for (int i = 0; i < N; ++i) acc_s[warp][lane + 32 * i] = acc[i];
  __syncthreads();
  float M = -INFINITY, L = 0.f;
  for (int y = 0; y < 4; ++y) M = fmaxf(M, ml_s[y].x);
  for (int y = 0; y < 4; ++y) L += weight_of(ml_s[y].x, M) * ml_s[y].y;
  const float inv = L == 0.f ? 0.f : 1.f / L;
  for (int d = 2 * threadIdx.x; d < a.kv.D; d += 256) {
    float o0 = 0.f, o1 = 0.f;
    for (int y = 0; y < 4; ++y) {
      const float c = weight_of(ml_s[y].x, M);
      o0 += c * acc_s[y][d];
      o1 += c * acc_s[y][d + 1];
    }
    store_out(a, t, hq, d, o0 * inv, o1 * inv);
  }
  if (threadIdx.x == 0) store_lse(a, t, hq, M, L);
}

// ------------------------------------------------------------------ host side ---
int padded(int D) { return (D + 63) / 64 * 64; }
// 8-head column tiles of a warp: two where the group needs them and the
// accumulators (2 * DP * tiles / 32 registers a lane and head pair) leave room.
int head_tiles(int DP, int G) { return DP <= 128 && G > 8 ? 2 : 1; }

struct Shape {
  int DP, NT, warps_h_log2, block_heads, blocks;
};

Shape shape_of(int D, int G) {
  Shape s;
  s.DP = padded(D);
  s.NT = head_tiles(s.DP, G);
  const int H = 8 * s.NT;
  s.warps_h_log2 = G > 2 * H ? 2 : G > H ? 1 : 0;
  s.block_heads = H << s.warps_h_log2;
  s.blocks = (G + s.block_heads - 1) / s.block_heads;
  return s;
}

size_t part_o_bytes(const Shape& s) { return static_cast<size_t>(kMaxWorkers) * 2 * s.block_heads * s.DP * sizeof(float); }
size_t part_ml_bytes(const Shape& s) { return static_cast<size_t>(kMaxWorkers) * 2 * s.block_heads * sizeof(float2); }

template <int FMT, int DP, int NT>
ft_status launch(AttnArgs& a, cudaStream_t s) {
  using X = Deal<FMT, DP>;
  static std::atomic<int> resident{0};  // CTAs an SM holds
  int r = resident.load(std::memory_order_relaxed);
  if (r == 0) {
    if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&r, attend_kernel<FMT, DP, NT>, kWarps * 32, 0) != cudaSuccess || r < 1)
      return fail(FT_ERR_CUDA, "attn_decode: %s", cudaGetErrorString(cudaGetLastError()));
    resident.store(r, std::memory_order_relaxed);
  }
  a.tile = 16 * X::U * (kWarps >> a.warps_h_log2);
  const int64_t longest = a.window > 0 && a.window < a.most ? a.window + 15 : a.most;
  const int64_t most_tiles = (longest + a.tile - 1) / a.tile * a.units * a.T;
  int64_t workers = static_cast<int64_t>(device_sm_count()) * r;
  if (workers > kMaxWorkers) workers = kMaxWorkers;
  if (workers > most_tiles) workers = most_tiles;
  a.workers = static_cast<int>(workers);
  attend_kernel<FMT, DP, NT><<<a.workers, kWarps * 32, 0, s>>>(a);
  ft_status st = launch_check("attn_decode");
  if (st != FT_OK) return st;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(a.T) * a.Hq);
  cfg.blockDim = dim3(128);
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  cudaLaunchKernelEx(&cfg, join_kernel<DP>, a);
  return launch_check("attn_decode join");
}

template <int FMT>
ft_status launch_shape(AttnArgs& a, const Shape& sh, cudaStream_t s) {
  switch (sh.DP) {
    case 64: return sh.NT == 2 ? launch<FMT, 64, 2>(a, s) : launch<FMT, 64, 1>(a, s);
    case 128: return sh.NT == 2 ? launch<FMT, 128, 2>(a, s) : launch<FMT, 128, 1>(a, s);
    case 192: return launch<FMT, 192, 1>(a, s);
    default: return launch<FMT, 256, 1>(a, s);
  }
}

bool attn_shape_ok(int32_t T, int32_t Hq, int32_t Hkv, int32_t D) {
  return T >= 0 && T <= 65535 && Hq > 0 && Hkv > 0 && Hq % Hkv == 0 && D >= 16 && D <= 256 && D % 16 == 0 &&
         static_cast<int64_t>(T) * Hq < (1ll << 31);
}

}  // namespace
}  // namespace ft

using namespace ft;

extern "C" {

size_t ft_attn_decode_workspace(int32_t T, int32_t Hq, int32_t Hkv, int32_t D) {
  if (!attn_shape_ok(T, Hq, Hkv, D)) return 0;
  const Shape s = shape_of(D, Hq / Hkv);
  return part_o_bytes(s) + part_ml_bytes(s);
}

ft_status ft_attn_decode(const ft_kv_cache* cache_host, const ft_rows* q_host, int32_t T, int32_t Hq, int32_t dtype,
                         const ft_page_table* table_host, const int32_t* seq, const int32_t* lens, float scale,
                         int32_t window, const ft_rows* out_host, int32_t out_dtype, float* lse, void* ws,
                         size_t ws_bytes, int32_t* dev_status, void* stream) {
  const char* what = "attn_decode";
  AttnArgs a = {};
  ft_status st;
  if ((st = kv_view(what, cache_host, table_host, seq, T, &a.kv)) != FT_OK) return st;
  const int32_t Hkv = cache_host->Hkv, fmt = cache_host->fmt;
  FT_REQUIRE(attn_shape_ok(T, Hq, Hkv, cache_host->D), "%s: T %d, Hq %d over %d key heads", what, T, Hq, Hkv);
  FT_REQUIRE(dtype == FT_DT_BF16 || dtype == FT_DT_F16, "%s: dtype %d", what, dtype);
  FT_REQUIRE(!(fmt == FT_KV_BF16 && dtype != FT_DT_BF16) && !(fmt == FT_KV_F16 && dtype != FT_DT_F16),
             "%s: a 16-bit cache takes queries of its own type", what);
  FT_REQUIRE(out_dtype == dtype || out_dtype == FT_DT_F32, "%s: out_dtype %d", what, out_dtype);
  FT_REQUIRE(isfinite(scale), "%s: scale is not finite", what);
  FT_REQUIRE(window >= 0, "%s: window %d", what, window);
  if (T == 0) return FT_OK;
  FT_REQUIRE(lens != nullptr, "%s: lens is NULL", what);
  if ((st = check_rows(what, "q", q_host, 8)) != FT_OK) return st;
  if ((st = check_rows(what, "out", out_host, out_dtype == FT_DT_F32 ? 4 : 8)) != FT_OK) return st;
  FT_REQUIRE(ws != nullptr && reinterpret_cast<uintptr_t>(ws) % 256 == 0, "%s: ws must be 256-byte aligned", what);
  const size_t need = ft_attn_decode_workspace(T, Hq, Hkv, cache_host->D);
  FT_REQUIRE(ws_bytes >= need, "%s: ws of %zu bytes, %zu needed", what, ws_bytes, need);
  const Shape sh = shape_of(cache_host->D, Hq / Hkv);
  a.q = static_cast<const uint16_t*>(q_host->base);
  a.q_tok = q_host->token_stride;
  a.q_head = q_host->head_stride;
  a.out = out_host->base;
  a.out_tok = out_host->token_stride;
  a.out_head = out_host->head_stride;
  a.lse = lse;
  a.lens = lens;
  a.part_o = static_cast<float*>(ws);
  a.part_ml = reinterpret_cast<float2*>(static_cast<uint8_t*>(ws) + part_o_bytes(sh));
  a.scale_log2 = scale * 1.4426950408889634f;
  a.window = window;
  a.T = T;
  a.Hq = Hq;
  a.G = Hq / Hkv;
  a.blocks = sh.blocks;
  a.units = Hkv * sh.blocks;
  a.warps_h_log2 = sh.warps_h_log2;
  a.block_heads = sh.block_heads;
  // token positions stay well inside 31 bits (a tile past the last is computed)
  const int64_t most = static_cast<int64_t>(table_host->max_pages) * cache_host->page_size;
  a.most = static_cast<int32_t>(most < (1ll << 31) - 4096 ? most : (1ll << 31) - 4096);
  a.q_f16 = dtype == FT_DT_F16;
  a.out_dtype = out_dtype;
  a.two_terms = out_dtype == FT_DT_F32;
  a.status = dev_status;
  cudaStream_t s = as_stream(stream);
  switch (fmt) {
    case FT_KV_BF16: return launch_shape<FT_KV_BF16>(a, sh, s);
    case FT_KV_F16: return launch_shape<FT_KV_F16>(a, sh, s);
    case FT_KV_E4M3: return launch_shape<FT_KV_E4M3>(a, sh, s);
    default: return launch_shape<FT_KV_NVFP4>(a, sh, s);
  }
}

}  // extern "C"
