// attn.cu -- attention of one new token a row over the paged key-value cache.
//
// For each row t and query head h:  x_j = scale q.k_j,  o = sum_j e^(x_j - m) v_j / sum_j e^(x_j - m)
// over the row's tokens j, in one pass with a running maximum m.  Every cached
// byte is read once and used by the G = Hq / Hkv query heads of its key head:
// 4 G flops a byte pair, far below the tensor cores' ridge, so the kernel is
// bound by HBM and everything is arranged around loads in flight.
//
// Layout of the work in a warp.  A warp works alone on steps of 16 or 32
// tokens: one lane a token looks its page up, and 16-byte asynchronous copies
// (any pages and strides; masked tokens become zeros) bring the rows into the
// warp's own ring in shared memory, several steps ahead and across the ends of
// units, so that loads stay in flight while the warp computes.  Keys become
// the A operand of mma.m16n8k16 (16 tokens x 16 channels, S^T = K Q^T) and
// values that of the second product (16 channels x 16 tokens, O^T = V^T P^T):
// the order of a contracted index is free as long as both operands agree, so a
// lane reads 16 contiguous bytes of a row and its elements are dealt to the
// fragments' places by renaming registers (keys) or by one byte permute a
// register (values, whose contracted index runs over tokens).  With tokens and
// channels on the 16-row side, 8 query heads fill the 8-column side.  P^T goes
// from accumulator to operand layout by movmatrix.  mma.sync and not tcgen05:
// 8- and 4-bit rows have to pass through registers to become 16-bit operands,
// and the tensor work is a small part of the time.  Copies by lanes and not by
// TMA: row gathers and bulk copies take their operands from uniform registers,
// so a warp that starts one for every four rows runs a loop of some 15
// instructions for each; measured, that cost more than it saved (4-bit rows,
// 64 rows up to 16384 tokens: 231 us against 186 us with loads into registers).
//
// Order of tokens.  Place r = 0..7 of the contracted index holds token r / 2
// (r even) or 4 + r / 2 (r odd) of its 8, so that a lane quarter's value rows
// are q, q + 4, q + 8, q + 12 and the swizzles below keep every read of shared
// memory free of bank conflicts.  Key rows and notes lie in the places' order,
// value rows in the tokens'.
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
#ifndef FT_TS_MIN
#define FT_TS_MIN 128
#endif
#ifndef FT_S3
#define FT_S3 3
#endif
#ifndef FT_C4
#define FT_C4 1
#endif
constexpr int kSmemSm = 227 * 1024;  // of an SM, for its CTAs' dynamic shared memory
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
  int2* shared_by;  // [row][unit] the first and the last worker of a unit that crossed shares; (1, 0) of any other
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

// The four E4M3 codes of a word as two f16 pairs.
__device__ __forceinline__ void e4m3x4(uint32_t w, uint32_t& lo, uint32_t& hi) {
  asm("{\n .reg .b16 a, b;\n mov.b32 {a, b}, %2;\n cvt.rn.f16x2.e4m3x2 %0, a;\n cvt.rn.f16x2.e4m3x2 %1, b;\n}"
      : "=r"(lo), "=r"(hi)
      : "r"(w));
}

// N words (1, 2 or 4) of shared memory.
template <int N>
__device__ __forceinline__ void load_words(uint32_t p, uint32_t (&w)[N]) {
  if constexpr (N == 4)
    asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]) : "r"(p));
  else if constexpr (N == 2)
    asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(w[0]), "=r"(w[1]) : "r"(p));
  else
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(w[0]) : "r"(p));
}

// 16 bytes from global to shared memory, past L1; `bytes` (16 or 0) of them read, the rest zeros.
__device__ __forceinline__ void copy16(uint32_t dst, const uint8_t* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copy16_or_zero(uint32_t dst, const uint8_t* src, uint32_t bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}

constexpr int gcd(int a, int b) { return b == 0 ? a : gcd(b, a % b); }

// How a format's rows are cut, for heads padded to DP channels (channels past
// D read zeros).  Keys: piece p of a row gives lane quarter q the EK channels
// p*4*EK + q*EK..; values: piece p gives lane group g the EV channels
// p*8*EV + g*EV...
template <int FMT, int DP, int NT>
struct Deal {
  static constexpr bool kQuant = FMT == FT_KV_E4M3 || FMT == FT_KV_NVFP4;
  static constexpr bool kBlocks = FMT == FT_KV_NVFP4;
  static constexpr bool kF16 = FMT != FT_KV_BF16;  // operand type of the products
  static constexpr int EK = !kQuant ? 8 : !kBlocks ? 16 : DP % 128 == 0 ? 32 : 16;
  static constexpr int EV = !kQuant ? 8 : !kBlocks ? (DP % 128 == 0 ? 16 : 8) : DP % 256 == 0 ? 32 : DP % 128 == 0 ? 16 : 8;
  static constexpr int NK = DP / (4 * EK), NV = DP / (8 * EV);
  static constexpr int bits = !kQuant ? 16 : kBlocks ? 4 : 8;
  static constexpr int WK = EK * bits / 32, WV = EV * bits / 32;  // words of a piece
  static constexpr int MT = DP / 16, H = 8 * NT;
  static constexpr int RB = DP * bits / 8;          // bytes of a row in shared memory
  static constexpr int PK = WK * 4, PV = WV * 4;    // bytes of a piece
  static constexpr bool kSwap = RB % 128 == 0;      // keys: odd places have 64-byte halves swapped
  static constexpr int KP = kSwap ? 2 : 1;
  static_assert(!kSwap || PK == 16, "");
  __device__ static constexpr int key_swizzle(int place) { return kSwap ? (place & 1) << 6 : 0; }
  __device__ static constexpr int value_swizzle(int token) {
    return PV == 16 ? (token & 3) << 5 : PV == 8 ? ((token >> 1) & 1) << 5 : 0;
  }
  // A step: TS tokens.
  static constexpr int TS = RB >= FT_TS_MIN ? 16 : 32;
  static constexpr int U = TS / 16;
  static constexpr int kSide = TS * RB;          // keys, or values, of a step
  // The copies of a step: chunk i = 32 c + lane of a side is row i / CPR, bytes 16 (i % CPR)..;
  // both repeat every CY copies, CR rows further on.
  static constexpr int CPR = RB / 16, kCopies = TS * CPR / 32;
  static constexpr int CY = CPR / gcd(32, CPR), CR = 32 * CY / CPR;
  static_assert(kCopies % CY == 0, "");
  // Beside a slot's rows, as copied: the words that hold the tokens' exponent
  // bytes (keys, then values), and the block scales (keys, then values).
  static constexpr int NBK = DP / 16, VS = TS + 4;
  static constexpr int kRawBlk = kBlocks ? TS * NBK : 0;
  static constexpr int kRaw = kQuant ? 2 * TS * 4 + 2 * kRawBlk : 0;
  // Once a warp, worked out when the step's turn comes: per place (key factor,
  // value exponent, 2^-value exponent, -), and the block scales as f16 (keys
  // [place][block], values [block][place]).
  static constexpr int kTok = kQuant ? TS * 16 : 0;
  static constexpr int kKeyBlk = kBlocks ? TS * NBK * 2 : 0, kValBlk = kBlocks ? NBK * VS * 2 : 0;
  static constexpr int kNotes = kTok + kKeyBlk + kValBlk;
  static constexpr uint32_t kFull = TS == 32 ? 0xffffffffu : (1u << (TS & 31)) - 1;
  // The merge of the warps takes two warps' sums at a time.
  static constexpr int kMerge = (MT * NT * 4 + NT * 4) * 32 * 4;
  // Slots of a warp's ring with so many CTAs an SM, and the choice of both.
  static constexpr int slots(int ctas) {
    const int n = ((kSmemSm / ctas - 1152 - 2 * kMerge) / kWarps - kNotes) / (2 * kSide + kRaw);
    return n < 8 ? n : 8;
  }
  static constexpr int kCtas = FT_C4 && kQuant && NT == 1 && DP <= 128 && slots(4) >= 2 ? 4 : slots(3) >= FT_S3 ? 3 : slots(2) >= 2 ? 2 : 1;
  static constexpr int S = slots(kCtas);
  static_assert(S >= 2, "");
  static constexpr int kSlot = 2 * kSide + kRaw;
  static constexpr int kRing = kWarps * S * kSlot;
  static constexpr int kSmem = 128 + kRing + kWarps * kNotes + 2 * kMerge;
  static_assert(kSlot % 128 == 0 && kNotes % 16 == 0 && 3 * S <= 32, "");
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

// A maximum over nothing: finite, so that 2^(-inf - kLowest) and 2^(kLowest - m) are 0 and not NaN.
constexpr float kLowest = -3.0e38f;
__device__ __forceinline__ float weight_of(float m, float M) { return exp2_approx(m - M); }

// The place of a token among its step's (see the order of tokens above), and the token of a place.
__device__ __forceinline__ constexpr int place_of(int t) { return (t & ~7) + 2 * (t & 3) + ((t >> 2) & 1); }
__device__ __forceinline__ constexpr int token_at(int r) { return (r & ~7) + 4 * (r & 1) + ((r >> 1) & 3); }

// A warp's way through its CTA's share of the line, unit by unit.
struct Walk {
  int t, at, left;   // row, place in the row's line, tiles left in the share
  int unit, tile0;   // the unit, and its first tile in this share
  int seq;           // the row's sequence
  int first, base, stop;  // tokens: the first that counts, this warp's next step's, the end
  bool whole;        // the share holds all of the unit
  int rest;          // the unit's tiles past the share

  // The next unit that the share touches; false at the share's end.  A row of
  // a bad sequence has no steps.
  __device__ __forceinline__ bool next(const AttnArgs& a, int offset) {
    if (left == 0) return false;
    RowSpan s = span_of(a, t);
    while (at >= s.tiles * a.units) {
      at -= s.tiles * a.units;
      s = span_of(a, ++t);
    }
    unit = at / s.tiles;
    tile0 = at - unit * s.tiles;
    const int n = min(s.tiles - tile0, left);
    at += n;
    left -= n;
    whole = n == s.tiles;
    rest = s.tiles - tile0 - n;
    seq = kv_seq(a.kv, t);
    first = s.first;
    base = s.begin + tile0 * a.tile + offset;
    stop = min(s.len, s.begin + (tile0 + n) * a.tile);
    if (static_cast<uint32_t>(seq) >= a.kv.n_seqs) {
      record_status(a.status, FT_ERR_BAD_ID);
      stop = 0;
    }
    return true;
  }
};

// The side of a warp that fills its ring, ahead of the side that computes.  A
// page is read one step before its use.
template <typename X>
struct Feeder {
  Walk walk;
  bool more, live;          // a step is prepared; the lane's token counts
  int32_t page;             // the token's page
  uint32_t place;           // and its place in it
  const int32_t* table;     // the unit's sequence's pages
  uint32_t head_row;        // the unit's key head
  uint32_t at;              // the slot to fill next
  uint32_t past;            // of the last steps, three bits each: the lane's token had a row, and that modulo 4
  // the lane's part of the copies, the same in every step (see Deal): source
  // chunk, and places in the keys' and the values' side of a slot
  const uint8_t* src[2][X::CY];
  uint32_t kdst[X::CY], vdst[X::CY];

  __device__ __forceinline__ void init(const AttnArgs& a, uint32_t ring, int lane) {
#pragma unroll
    for (int c = 0; c < X::CY; ++c) {
      const int row = (c * 32 + lane) / X::CPR, chunk = (c * 32 + lane) % X::CPR;
      src[0][c] = a.kv.data[0] + chunk * 16;
      src[1][c] = a.kv.data[1] + chunk * 16;
      kdst[c] = place_of(row) * X::RB + ((chunk * 16) ^ X::key_swizzle(place_of(row)));
      vdst[c] = X::kSide + row * X::RB + ((chunk * 16) ^ X::value_swizzle(row));
    }
    at = ring;
    past = 0;
  }

  __device__ __forceinline__ void prepare(const AttnArgs& a, int offset, int step, int lane) {
    while (walk.base >= walk.stop) {
      if (!walk.next(a, offset)) {
        more = false;
        return;
      }
      table = a.kv.pages + walk.seq * a.kv.table_stride;
      head_row = static_cast<uint32_t>(walk.unit / a.blocks) * a.kv.at.head_stride;
    }
    more = true;
    const int tok = walk.base + lane;
    live = lane < X::TS && tok >= walk.first && tok < walk.stop;
    if (live) {
      const uint32_t p = fast_div(tok, a.kv.at.by_page);
      place = tok - p * a.kv.at.page_size;
      page = table[p];
    }
    walk.base += step;
  }

  // The block scales of the lane's token into the slot.  Rows of an odd number
  // of byte pairs are not word-aligned: read and stored.
  __device__ __forceinline__ void copy_blocks(const AttnArgs& a, uint32_t row, int lane) {
    if constexpr (X::kBlocks) {
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const uint8_t* from = a.kv.block[j] + static_cast<uint64_t>(row) * (a.kv.D >> 4);
        const uint32_t to = at + 2 * X::kSide + 2 * X::TS * 4 + j * X::kRawBlk + lane * X::NBK;
        if (a.kv.D == X::NBK * 16) {
          if constexpr (X::NBK == 16) {
            copy16(to, from);
          } else if constexpr (X::NBK == 8) {
            asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(to), "l"(from) : "memory");
          } else {
#pragma unroll
            for (int w = 0; w < X::NBK / 4; ++w)
              asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(to + 4 * w), "l"(from + 4 * w) : "memory");
          }
        } else {
#pragma unroll
          for (int w = 0; w < X::NBK / 2; ++w) {
            const uint16_t v = 32 * w < a.kv.D ? *reinterpret_cast<const uint16_t*>(from + 2 * w) : 0;
            asm volatile("st.shared.u16 [%0], %1;" ::"r"(to + 2 * w), "h"(v) : "memory");
          }
        }
      }
    }
  }

  // The notes of the step in slot `slot`, S steps after its issue: one lane a token.
  __device__ __forceinline__ void put_notes(uint32_t slot, uint32_t notes, int lane) const {
    if constexpr (X::kQuant) {
      if (lane < X::TS) {
        const uint32_t was = past >> (3 * (X::S - 1));
        const bool ok = (was & 4) != 0;
        const uint32_t raw = slot + 2 * X::kSide, sh = (was & 3) * 8;
        uint32_t kw, vw;
        asm volatile("ld.shared.u32 %0, [%1];" : "=r"(kw) : "r"(raw + lane * 4));
        asm volatile("ld.shared.u32 %0, [%1];" : "=r"(vw) : "r"(raw + X::TS * 4 + lane * 4));
        // exponent bytes as writers store them; others are held to 2^-100 .. 2^123
        const uint32_t kb = min(max((kw >> sh) & 0xffu, 27u), 250u), vb = min(max((vw >> sh) & 0xffu, 27u), 250u);
        const float ks = ok ? __uint_as_float(kb << 23) : 0.f;
        const float ev = ok ? static_cast<float>(static_cast<int>(vb) - 127) : -INFINITY;
        const float iv = ok ? __uint_as_float((254u - vb) << 23) : 0.f;
        const uint32_t pl = place_of(lane);
        asm volatile("st.shared.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(notes + pl * 16), "f"(ks), "f"(ev), "f"(iv), "f"(0.f)
                     : "memory");
        if constexpr (X::kBlocks) {
          const uint32_t ka = notes + X::kTok + pl * (X::NBK * 2);
          const uint32_t va = notes + X::kTok + X::kKeyBlk + pl * 2;
#pragma unroll
          for (int w = 0; w < X::NBK / 4; ++w) {
            uint32_t kq, vq;
            const uint32_t from = raw + 2 * X::TS * 4 + lane * X::NBK + w * 4;
            asm volatile("ld.shared.u32 %0, [%1];" : "=r"(kq) : "r"(from));
            asm volatile("ld.shared.u32 %0, [%1];" : "=r"(vq) : "r"(from + X::kRawBlk));
            uint32_t k2[2], v2[2];
            e4m3x4(ok ? kq : 0, k2[0], k2[1]);
            e4m3x4(ok ? vq : 0, v2[0], v2[1]);
            asm volatile("st.shared.v2.u32 [%0], {%1, %2};" ::"r"(ka + w * 8), "r"(k2[0]), "r"(k2[1]) : "memory");
#pragma unroll
            for (int i = 0; i < 4; ++i)
              asm volatile("st.shared.u16 [%0], %1;" ::"r"(va + (4 * w + i) * (X::VS * 2)),
                           "h"(static_cast<uint16_t>(v2[i >> 1] >> (16 * (i & 1))))
                           : "memory");
          }
        }
      }
      __syncwarp();
    }
  }

  // The tokens of the oldest step that counts, one bit each.
  __device__ __forceinline__ uint32_t mask() const { return __ballot_sync(kAll, (past >> (3 * (X::S - 1)) & 4) != 0); }

  // Starts the prepared step's copies into its slot.  One group of copies a
  // call, whether it has any or not.
  __device__ __forceinline__ void issue(const AttnArgs& a, uint32_t ring, int lane) {
    __syncwarp();  // every lane has finished reading the slot
    past <<= 3;
    if (more) {
      uint32_t row = kNoRow;
      if (live) {
        row = kv_row(a.kv.at, page, place);
        if (row == kNoRow)
          record_status(a.status, FT_ERR_BAD_ID);
        else
          row += head_row;
      }
      const bool has_row = row != kNoRow;
      if (has_row) past |= 4 | (row & 3);
      const uint32_t counts = __ballot_sync(kAll, has_row);
      // Rows (c / CY) * CR further on move a lane's places by constants: the
      // order of places and the swizzles only rearrange and join bits, and the
      // rows of one period are the low bits.
      if (counts == X::kFull && a.kv.row_bytes == X::RB) {
#pragma unroll
        for (int c = 0; c < X::kCopies; ++c) {
          const int cy = c % X::CY, on = c / X::CY * X::CR;
          const uint32_t n = __shfl_sync(kAll, row, (cy * 32 + lane) / X::CPR + on);
          copy16(at + (kdst[cy] ^ X::key_swizzle(place_of(on))) + place_of(on) * X::RB,
                 src[0][cy] + static_cast<uint64_t>(n) * X::RB);
          copy16(at + (vdst[cy] ^ X::value_swizzle(on)) + on * X::RB, src[1][cy] + static_cast<uint64_t>(n) * X::RB);
        }
      } else {
#pragma unroll
        for (int c = 0; c < X::kCopies; ++c) {
          const int cy = c % X::CY, on = c / X::CY * X::CR;
          const uint32_t n = __shfl_sync(kAll, row, (cy * 32 + lane) / X::CPR + on);
          const bool ok = n != kNoRow && (cy * 32 + lane) % X::CPR * 16 < a.kv.row_bytes;
          const uint64_t off = ok ? static_cast<uint64_t>(n) * a.kv.row_bytes : 0;
          copy16_or_zero(at + (kdst[cy] ^ X::key_swizzle(place_of(on))) + place_of(on) * X::RB,
                         ok ? src[0][cy] + off : a.kv.data[0], ok ? 16 : 0);
          copy16_or_zero(at + (vdst[cy] ^ X::value_swizzle(on)) + on * X::RB, ok ? src[1][cy] + off : a.kv.data[1],
                         ok ? 16 : 0);
        }
      }
      if constexpr (X::kQuant) {
        if (has_row) {
          // the aligned words around the exponent bytes
          const uint32_t to = at + 2 * X::kSide + lane * 4;
          asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(to), "l"(a.kv.scale[0] + (row & ~3u)) : "memory");
          asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(to + X::TS * 4), "l"(a.kv.scale[1] + (row & ~3u))
                       : "memory");
          copy_blocks(a, row, lane);
        }
      }
      at += X::kSlot;
      if (at == ring + X::S * X::kSlot) at = ring;
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  }
};

// The weights are rescaled when a score exceeds the running reference by this
// much (in powers of two), not at every new maximum: 2^4 leaves p far inside f16.
constexpr float kSlack = 4.f;

template <typename X, bool TWO, int NT>
__device__ __forceinline__ void add_values(uint32_t at, uint32_t vnotes, int u, int g, int q,
                                           const uint32_t (&hi)[NT][2], const uint32_t (&lo)[NT][2],
                                           float (&acc)[X::MT][NT][4]) {
  const auto step = [&](int mt, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3) {
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      mma<X::kF16>(acc[mt][n], a0, a1, a2, a3, hi[n][0], hi[n][1]);
      if (TWO) mma<X::kF16>(acc[mt][n], a0, a1, a2, a3, lo[n][0], lo[n][1]);
    }
  };
#pragma unroll
  for (int p = 0; p < X::NV; ++p) {
    uint32_t v[4][X::WV];
#pragma unroll
    for (int r = 0; r < 4; ++r)
      load_words(at + p * (8 * X::PV) + (16 * u + 4 * r) * X::RB, v[r]);
    const int m0 = p * (X::EV / 2);
    uint32_t b0 = 0, b1 = 0;  // block scales of the tokens q, q + 4 and q + 8, q + 12
#pragma unroll
    for (int w = 0; w < X::WV; ++w) {
      const uint32_t t0 = v[0][w], t1 = v[1][w], t2 = v[2][w], t3 = v[3][w];
      if constexpr (!X::kQuant) {
        step(m0 + w, __byte_perm(t0, t1, 0x5410), __byte_perm(t0, t1, 0x7632), __byte_perm(t2, t3, 0x5410),
             __byte_perm(t2, t3, 0x7632));
      } else if constexpr (!X::kBlocks) {
        // bytes of two tokens side by side, then two conversions a word
        uint32_t f[8];
        e4m3x4(__byte_perm(t0, t1, 0x5140), f[0], f[1]);
        e4m3x4(__byte_perm(t2, t3, 0x5140), f[2], f[3]);
        e4m3x4(__byte_perm(t0, t1, 0x7362), f[4], f[5]);
        e4m3x4(__byte_perm(t2, t3, 0x7362), f[6], f[7]);
        step(m0 + 2 * w, f[0], f[1], f[2], f[3]);
        step(m0 + 2 * w + 1, f[4], f[5], f[6], f[7]);
      } else {
        if (w % 2 == 0) {
          const int block = X::EV >= 16 ? p * (X::EV / 2) + g * (X::EV / 16) + w / 2 : p * 4 + (g >> 1);
          const uint32_t na = vnotes + block * (X::VS * 2) + (16 * u + 2 * q) * 2;
          asm volatile("ld.shared.u32 %0, [%1];" : "=r"(b0) : "r"(na));
          asm volatile("ld.shared.u32 %0, [%1];" : "=r"(b1) : "r"(na + 16));
        }
        // nibbles of two tokens side by side: even elements, odd elements
        const uint32_t m = 0x0f0f0f0fu;
        uint32_t e0[4], o0[4], e1[4], o1[4];
        e2m1x8((t0 & m) | ((t1 & m) << 4), e0);
        e2m1x8(((t0 >> 4) & m) | (t1 & ~m), o0);
        e2m1x8((t2 & m) | ((t3 & m) << 4), e1);
        e2m1x8(((t2 >> 4) & m) | (t3 & ~m), o1);
#pragma unroll
        for (int i = 0; i < 4; ++i)
          step(m0 + 4 * w + i, mul_f16x2(e0[i], b0), mul_f16x2(o0[i], b0), mul_f16x2(e1[i], b1), mul_f16x2(o1[i], b1));
      }
    }
  }
}

template <int FMT, int DP, int NT>
__global__ void __launch_bounds__(kWarps * 32, Deal<FMT, DP, NT>::kCtas)
    attend_kernel(const __grid_constant__ AttnArgs a) {
  using X = Deal<FMT, DP, NT>;
  constexpr int U = X::U, MT = X::MT, H = X::H, S = X::S;
  extern __shared__ uint8_t smem_raw[];
  pdl_launch_dependents();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, q = lane & 3;
  const int wh = warp & ((1 << a.warps_h_log2) - 1), wt = warp >> a.warps_h_log2;
  const int warps_t = kWarps >> a.warps_h_log2;

  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 127) & ~uintptr_t(127));
  const uint32_t ring = smem_u32(smem) + warp * (S * X::kSlot);
  const uint32_t note = smem_u32(smem) + X::kRing + warp * X::kNotes;
  float* merge = reinterpret_cast<float*>(smem + X::kRing + kWarps * X::kNotes);

  // this CTA's share of the line, and the row it begins in
  const int64_t total = tiles_before(a, a.T, lane) * a.units;
  const int64_t share = split_share(total, a.workers);
  const int64_t from = blockIdx.x * share;
  // rows that see nothing
  for (int t = blockIdx.x; t < a.T; t += gridDim.x)
    if (span_of(a, t).tiles == 0) {
      for (int i = threadIdx.x; i < a.Hq * (a.kv.D / 2); i += kWarps * 32) {
        const int h = i / (a.kv.D / 2), d = 2 * (i - h * (a.kv.D / 2));
        store_out(a, t, h, d, 0.f, 0.f);
        if (d == 0) store_lse(a, t, h, -INFINITY, 0.f);
      }
      for (int i = threadIdx.x; i < a.units; i += kWarps * 32) a.shared_by[t * a.units + i] = make_int2(1, 0);
    }
  if (from >= total) return;
  Walk walk;
  walk.left = static_cast<int>(from + share < total ? share : total - from);
  {
    int64_t row_at = 0;  // the row's first number
    for (int t0 = 0;; t0 += 32) {
      const int64_t n = t0 + lane < a.T ? static_cast<int64_t>(span_of(a, t0 + lane).tiles) * a.units : 0;
      int64_t upto = n;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int64_t y = __shfl_up_sync(kAll, upto, o);
        if (lane >= o) upto += y;
      }
      const uint32_t past = __ballot_sync(kAll, row_at + upto > from);
      if (past) {
        const int i = __ffs(past) - 1;
        walk.t = t0 + i;
        walk.at = static_cast<int>(from - row_at - __shfl_sync(kAll, upto - n, i));
        break;
      }
      row_at += __shfl_sync(kAll, upto, 31);
    }
  }
  walk.base = walk.stop = 0;
  const int offset = wt * X::TS, step = X::TS * warps_t;

  Feeder<X> feed;
  feed.walk = walk;
  feed.init(a, ring, lane);
  feed.prepare(a, offset, step, lane);
#pragma unroll 1
  for (int i = 0; i < S; ++i) {
    feed.issue(a, ring, lane);
    if (feed.more) feed.prepare(a, offset, step, lane);
  }

  // places of the lane's pieces in a step's rows
  uint32_t koff[X::KP];
#pragma unroll
  for (int p = 0; p < X::KP; ++p) koff[p] = g * X::RB + ((p * 4 + q) * X::PK ^ X::key_swizzle(g));
  const uint32_t voff = q * X::RB + (g * X::PV ^ X::value_swizzle(q));

  uint32_t at = ring;  // the slot to read next
  while (walk.next(a, offset)) {
    const int t = walk.t;
    const int kv_head = walk.unit / a.blocks;
    const int head0 = (walk.unit - kv_head * a.blocks) * a.block_heads;  // of the key head's group

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
        constexpr int E = X::EK / 4;
        const int d = (st / E) * 4 * X::EK + q * X::EK + (st % E) * 4;
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
        m[n][i] = kLowest;
        l[n][i] = 0.f;
      }
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[mt][n][i] = 0.f;
    }

#pragma unroll 1
    for (; walk.base < walk.stop; walk.base += step) {
      asm volatile("cp.async.wait_group %0;" ::"n"(S - 1) : "memory");
      __syncwarp();
      feed.put_notes(at, note, lane);

      // s[u][n] = S^T of 16 tokens: (token g | g + 8) x (head 2q | 2q + 1)
      float s[U][NT][4];
#pragma unroll
      for (int u = 0; u < U; ++u) {
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int i = 0; i < 4; ++i) s[u][n][i] = 0.f;
#pragma unroll
        for (int p = 0; p < X::NK; ++p) {
          uint32_t f[2][X::EK / 2];  // 16-bit pairs of rows g and g + 8
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            uint32_t k[X::WK];
            load_words(at + (p / X::KP) * (X::KP * 4 * X::PK) + koff[p % X::KP] + (16 * u + 8 * r) * X::RB, k);
            if constexpr (!X::kQuant) {
#pragma unroll
              for (int w = 0; w < X::WK; ++w) f[r][w] = k[w];
            } else if constexpr (!X::kBlocks) {
#pragma unroll
              for (int w = 0; w < X::WK; ++w) e4m3x4(k[w], f[r][2 * w], f[r][2 * w + 1]);
            } else {
              uint32_t b2;  // the lane's block scales: one or two
              const uint32_t na = note + X::kTok + (16 * u + 8 * r + g) * (X::NBK * 2) + (p * 4 + q) * (X::EK / 8);
              if (X::EK == 32) {
                asm volatile("ld.shared.u32 %0, [%1];" : "=r"(b2) : "r"(na));
              } else {
                uint16_t b1;
                asm volatile("ld.shared.u16 %0, [%1];" : "=h"(b1) : "r"(na));
                b2 = b1;
              }
#pragma unroll
              for (int w = 0; w < X::WK; ++w) {
                uint32_t h[4];
                e2m1x8(k[w], h);
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
              mma<X::kF16>(s[u][n], f[0][2 * i], f[1][2 * i], f[0][2 * i + 1], f[1][2 * i + 1], qb[st][n][0],
                           qb[st][n][1]);
            }
        }
      }

      // scores in powers of two, with the value's exponent; masked tokens -inf
      float iv[U][2];
      bool more = false;
      const uint32_t mask = X::kQuant ? 0 : feed.mask();
      const bool part = !X::kQuant && mask != X::kFull;
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          float ks = 1.f, ev = 0.f, none;
          iv[u][r] = 1.f;
          if constexpr (X::kQuant)
            asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];"
                         : "=f"(ks), "=f"(ev), "=f"(iv[u][r]), "=f"(none)
                         : "r"(note + (16 * u + 8 * r + g) * 16));
          const bool ok = (mask >> token_at(16 * u + 8 * r + g)) & 1;
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              float& x = s[u][n][2 * r + i];
              x = X::kQuant ? fmaf(x * ks, mul[n][i], ev) : x * mul[n][i];
              if (part) x = ok ? x : -INFINITY;
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
      const bool two = !X::kF16 || a.two_terms;
#pragma unroll
      for (int u = 0; u < U; ++u) {
        uint32_t hi[NT][2], lo[NT][2];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            const float p0 = exp2_approx(s[u][n][2 * r] - m[n][0]), p1 = exp2_approx(s[u][n][2 * r + 1] - m[n][1]);
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
            if (two) {
              const float2 back = unpack16<X::kF16>(h);
              lo[n][r] = transpose8x8(pack16<X::kF16>(p0 - back.x, p1 - back.y));
            }
          }
        }
        const uint32_t vnotes = note + X::kTok + X::kKeyBlk;
        if (two)
          add_values<X, true, NT>(at + X::kSide + voff, vnotes, u, g, q, hi, lo, acc);
        else if constexpr (X::kF16)
          add_values<X, false, NT>(at + X::kSide + voff, vnotes, u, g, q, hi, lo, acc);
      }
      feed.issue(a, ring, lane);  // refills this slot
      if (feed.more) feed.prepare(a, offset, step, lane);
      at += X::kSlot;
      if (at == ring + S * X::kSlot) at = ring;
    }

    // The warps' sums meet in shared memory, half of them handing over at a
    // time.  A warp hands over in the place that it took over from before.
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        l[n][i] += __shfl_xor_sync(kAll, l[n][i], 4);
        l[n][i] += __shfl_xor_sync(kAll, l[n][i], 8);
        l[n][i] += __shfl_xor_sync(kAll, l[n][i], 16);
      }
    if (warps_t > 1) __syncthreads();  // the places are free of the unit before
    for (int half = warps_t >> 1; half > 0; half >>= 1) {
      float* place = merge + (half == 2 ? wt & 1 : a.warps_h_log2 ? wh : 1) * (X::kMerge / 4) + lane;
      if (wt >= half && wt < 2 * half) {
#pragma unroll
        for (int n = 0; n < NT; ++n) {
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            place[(n * 4 + i) * 32] = m[n][i];
            place[(n * 4 + 2 + i) * 32] = l[n][i];
          }
#pragma unroll
          for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int i = 0; i < 4; ++i) place[(NT * 4 + (mt * NT + n) * 4 + i) * 32] = acc[mt][n][i];
        }
      }
      __syncthreads();
      if (wt < half) {
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const float om = place[(n * 4 + i) * 32], ol = place[(n * 4 + 2 + i) * 32];
            const float top = fmaxf(m[n][i], om);
            const float x = weight_of(m[n][i], top), y = weight_of(om, top);
            m[n][i] = top;
            l[n][i] = l[n][i] * x + ol * y;
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
              float* o = place + (NT * 4 + (mt * NT + n) * 4) * 32;
              acc[mt][n][i] = acc[mt][n][i] * x + o[i * 32] * y;
              acc[mt][n][2 + i] = acc[mt][n][2 + i] * x + o[(2 + i) * 32] * y;
            }
          }
      }
    }
    if (threadIdx.x == 0 && walk.tile0 == 0) {
      const int first = blockIdx.x, last = first + static_cast<int>((walk.rest + share - 1) / share);
      a.shared_by[t * a.units + walk.unit] = walk.whole ? make_int2(1, 0) : make_int2(first, last);
    }
    if (wt == 0) {
      const int64_t part = static_cast<int64_t>(blockIdx.x) * 2 + (walk.tile0 == 0 ? 1 : 0);
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int h = wh * H + n * 8 + 2 * q + i;  // in the block
          if (h >= a.block_heads || head0 + h >= a.G) continue;
          const float M = m[n][i], L = l[n][i];
          const float inv = L == 0.f ? 0.f : 1.f / L;
#pragma unroll
          for (int mt = 0; mt < MT; ++mt) {
            const int d = (mt / (X::EV / 2)) * 8 * X::EV + g * X::EV + 2 * (mt % (X::EV / 2));
            if (!walk.whole)
              *reinterpret_cast<float2*>(a.part_o + (part * a.block_heads + h) * DP + d) =
                  make_float2(acc[mt][n][i], acc[mt][n][2 + i]);
            else if (d < a.kv.D)
              store_out(a, t, kv_head * a.G + head0 + h, d, acc[mt][n][i] * inv, acc[mt][n][2 + i] * inv);
          }
          if (g == 0) {
            if (walk.whole)
              store_lse(a, t, kv_head * a.G + head0 + h, M, L);
            else
              a.part_ml[part * a.block_heads + h] = make_float2(M, L);
          }
        }
    }
  }
}

// Adds the partial sums of unit blockIdx.x, if it crossed shares, in the
// workers' order.  A CTA takes kHeads heads of the block, 8 / kHeads warps a
// head (each every so-many-th partial): one head where few units have many
// partials each (one long row), eight otherwise.
template <int DP, int kHeads>
__global__ void __launch_bounds__(256) join_kernel(const __grid_constant__ AttnArgs a) {
  constexpr int N = DP / 64;           // channel pairs of a lane: 2 * lane + 64 i
  constexpr int kSpread = 8 / kHeads;  // warps of a head
  constexpr int kBatch = kHeads == 1 ? 8 : 2;  // partials in flight
  __shared__ float2 acc_s[kSpread > 1 ? 8 : 1][DP / 2];
  __shared__ float2 ml_s[8];
  // every CTA waits, whether it has something to add or not: work after this
  // grid must also come after attend_kernel
  pdl_wait();
  const int2 workers = a.shared_by[blockIdx.x];
  if (workers.y <= workers.x) return;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int h = blockIdx.y * kHeads + warp / kSpread;
  const int t = blockIdx.x / a.units, unit = blockIdx.x - t * a.units;
  const int kv_head = unit / a.blocks;
  const int hg = (unit - kv_head * a.blocks) * a.block_heads + h;  // in the key head's group
  const bool live = h < a.block_heads && hg < a.G;
  const int c0 = workers.x, c1 = workers.y;
  float m = kLowest, l = 0.f;
  float2 acc[N];
#pragma unroll
  for (int i = 0; i < N; ++i) acc[i] = make_float2(0.f, 0.f);
  for (int c = c0 + warp % kSpread; live && c <= c1; c += kBatch * kSpread) {
    float2 ml[kBatch], o[kBatch][N];
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      const int ck = c + k * kSpread;
      ml[k] = make_float2(kLowest, 0.f);
#pragma unroll
      for (int i = 0; i < N; ++i) o[k][i] = make_float2(0.f, 0.f);
      if (ck <= c1) {
        const int64_t slot = (static_cast<int64_t>(ck) * 2 + (ck == c0 ? 1 : 0)) * a.block_heads + h;
        ml[k] = a.part_ml[slot];
#pragma unroll
        for (int i = 0; i < N; ++i) o[k][i] = *reinterpret_cast<const float2*>(a.part_o + slot * DP + 2 * lane + 64 * i);
      }
    }
    float top = m;
#pragma unroll
    for (int k = 0; k < kBatch; ++k) top = fmaxf(top, ml[k].x);
    const float x = weight_of(m, top);
    m = top;
    l *= x;
#pragma unroll
    for (int i = 0; i < N; ++i) acc[i] = make_float2(acc[i].x * x, acc[i].y * x);
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      const float y = weight_of(ml[k].x, top);
      l += ml[k].y * y;
#pragma unroll
      for (int i = 0; i < N; ++i) {
        acc[i].x += o[k][i].x * y;
        acc[i].y += o[k][i].y * y;
      }
    }
  }
  if (kSpread > 1) {
    if (lane == 0) ml_s[warp] = make_float2(m, l);
#pragma unroll
    for (int i = 0; i < N; ++i) acc_s[warp][lane + 32 * i] = acc[i];
    __syncthreads();
    if (warp % kSpread != 0) return;
    const float own = m;
#pragma unroll
    for (int y = 0; y < kSpread; ++y) m = fmaxf(m, ml_s[warp + y].x);
    const float x = weight_of(own, m);
    l *= x;
#pragma unroll
    for (int i = 0; i < N; ++i) acc[i] = make_float2(acc[i].x * x, acc[i].y * x);
#pragma unroll
    for (int y = 1; y < kSpread; ++y) {
      const float w = weight_of(ml_s[warp + y].x, m);
      l += w * ml_s[warp + y].y;
#pragma unroll
      for (int i = 0; i < N; ++i) {
        acc[i].x += w * acc_s[warp + y][lane + 32 * i].x;
        acc[i].y += w * acc_s[warp + y][lane + 32 * i].y;
      }
    }
  }
  if (!live) return;
  const int hq = kv_head * a.G + hg;
  const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll
  for (int i = 0; i < N; ++i)
    if (2 * lane + 64 * i < a.kv.D) store_out(a, t, hq, 2 * lane + 64 * i, acc[i].x * inv, acc[i].y * inv);
  if (lane == 0) store_lse(a, t, hq, m, l);
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
  using X = Deal<FMT, DP, NT>;
  ft_status st = ensure_dyn_smem(reinterpret_cast<const void*>(attend_kernel<FMT, DP, NT>), X::kSmem, "attn_decode");
  if (st != FT_OK) return st;
  static std::atomic<int> resident{0};  // CTAs an SM holds
  int r = resident.load(std::memory_order_relaxed);
  if (r == 0) {
    if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&r, attend_kernel<FMT, DP, NT>, kWarps * 32, X::kSmem) != cudaSuccess ||
        r < 1)
      return fail(FT_ERR_CUDA, "attn_decode: %s", cudaGetErrorString(cudaGetLastError()));
    resident.store(r, std::memory_order_relaxed);
  }
  a.tile = X::TS * (kWarps >> a.warps_h_log2);
  const int64_t longest = a.window > 0 && a.window < a.most ? a.window + 15 : a.most;
  const int64_t most_tiles = (longest + a.tile - 1) / a.tile * a.units * a.T;
  int64_t workers = static_cast<int64_t>(device_sm_count()) * r;
  if (workers > kMaxWorkers) workers = kMaxWorkers;
  if (workers > most_tiles) workers = most_tiles;
  // positions in a row's line, and in a share, are 32-bit in the kernel
  if (most_tiles / a.T >= (1ll << 31) || most_tiles / workers >= (1ll << 31))
    return fail(FT_ERR_UNSUPPORTED, "attn_decode: page table too large");
  a.workers = static_cast<int>(workers);
  attend_kernel<FMT, DP, NT><<<a.workers, kWarps * 32, X::kSmem, s>>>(a);
  st = launch_check("attn_decode");
  if (st != FT_OK) return st;
  cudaLaunchConfig_t cfg = {};
  const bool long_rows = workers > 8ll * a.T * a.units;  // more than eight partials a unit on average
  cfg.gridDim = dim3(a.T * a.units, long_rows ? a.block_heads : a.block_heads / 8);
  cfg.blockDim = dim3(256);
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  cudaLaunchKernelEx(&cfg, long_rows ? join_kernel<DP, 1> : join_kernel<DP, 8>, a);
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
  return part_o_bytes(s) + part_ml_bytes(s) + static_cast<size_t>(T) * Hkv * s.blocks * sizeof(int2);
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
  a.shared_by = reinterpret_cast<int2*>(static_cast<uint8_t*>(ws) + part_o_bytes(sh) + part_ml_bytes(sh));
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
