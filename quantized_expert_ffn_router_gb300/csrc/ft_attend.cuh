// ft_attend.cuh -- attention of one new token a row over the paged key-value
// cache: the kernel, for one cache format a translation unit (attn_*.cu).
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
// Columns.  A warp's registers hold the sums of 16 heads of up to 128 channels,
// or of 8 wider ones.  Where a key head has more query heads, two or four warps
// side by side take them: they fill one ring together and meet once a step
// (64 heads over one of 128, 128 rows up to 16384 tokens, bf16: 137 us; 241
// with a ring for each warp).  Otherwise a CTA's four warps take different
// tokens, each with a ring of its own, and meet at a unit's end.  Two tiles of
// 8 heads in a warp beat two warps of one (16 rows up to 16384, 16 heads over
// each of 4 of 128, E4M3, one term a weight: 36 us and 47): rows are turned into
// operands once.
//
// Order of tokens.  Place r = 0..7 of the contracted index holds token r / 2
// (r even) or 4 + r / 2 (r odd) of its 8, so that a lane quarter's value rows
// are q, q + 4, q + 8, q + 12 and the swizzles below keep every read of shared
// memory free of bank conflicts.  Key rows and notes lie in the places' order,
// value rows in the tokens'.
//
// 8- and 4-bit rows: a key's power-of-two scale multiplies its score; a
// value's enters the running maximum, so that the weight that is rounded to
// f16 is p_j = 2^(x_j + ev_j - m) <= 2^15 whatever the scales are, and the sum
// of the softmax takes p_j 2^-ev_j in fp32.
//
// Split.  The tiles of all rows and key heads are numbered in one line and cut
// into equal shares, one a CTA (lengths are read on the device, so a captured
// graph serves any lengths).  A unit (row, head block) inside one share is
// written directly; one that crosses shares leaves partial sums that
// join_kernel adds in order.
//
// What it measured (GPU time in a graph, inputs beyond L2; HBM at 6.70 TB/s):
//   one row of 1000003 tokens, 32 heads over 4 of 128: bf16 299-302 us (the copy
//   rate), E4M3 168 us (92% of it), NVFP4 141 us (62%);
//   32 rows up to 8192 tokens, 32 heads over 8, bf16: 62.2 us (88%), E4M3 42
//   (66%), NVFP4 39 (40%);
//   64 rows up to 16384, 64 heads over 8, NVFP4: 109 us (58%).
// 16-bit rows are bound by HBM, 4-bit rows by instructions and their latency (60%
// of the issue slots, four warps a scheduler): of 403 warp instructions for 16
// tokens of one key head, 190 turn codes into operands (conversions, bytes taken
// out of words, block scales), 24 are products, and 20 or so are the weights'
// second term.
// Short work is bound by latency: about 4 us from the launch to the first rows
// in shared memory, 1.5-2 us for a unit's merge, 3 us for the join.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <math.h>

#include <atomic>

#include "ft_attn_args.cuh"

namespace ft {
namespace {

constexpr int kSmemSm = 227 * 1024;  // of an SM, for its CTAs' dynamic shared memory
constexpr uint32_t kAll = 0xffffffffu;

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

constexpr int log2_of(int n) { return n == 1 ? 0 : 1 + log2_of(n / 2); }
constexpr int gcd(int a, int b) { return b == 0 ? a : gcd(b, a % b); }

// How a format's rows are cut, for heads padded to DP channels (channels past
// D read zeros).  Keys: piece p of a row gives lane quarter q the EK channels
// p*4*EK + q*EK..; values: piece p gives lane group g the EV channels
// p*8*EV + g*EV...
// COLS: warps side by side over a block's heads.
template <int FMT, int DP, int NT, int COLS>
struct Deal {
  static constexpr int kFmt = FMT;
  static constexpr int kWarps = COLS == 1 ? 4 : COLS, kThreads = kWarps * 32;
  static constexpr int kWarpsT = COLS == 1 ? 4 : 1;  // warps side by side over tokens
  static constexpr int kRings = kWarpsT, kFill = 32 * COLS;  // threads that fill a ring
  static constexpr bool kQuant = FMT == FT_KV_E4M3 || FMT == FT_KV_NVFP4;
  static constexpr bool kBlocks = FMT == FT_KV_NVFP4;
  static constexpr bool kF16 = FMT != FT_KV_BF16;  // operand type of the products
  // How far the reference lies below the greatest score.  f16 weights reach
  // 2^(11 + kSlack), the top of its range, so that what rounds to nothing (f16's
  // steps end at 2^-24) is 2^-36 of the heaviest: with the heaviest at 1, a
  // token 18 nats above 16384 others took 6% of the norm from them.  bf16 has
  // fp32's range, in its values too: weights of 2^-24 keep the sums of 2^24
  // tokens of the largest values inside it.
  static constexpr int kLift = kF16 ? 11 : -24;
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
  // A step: TS tokens, 2 to 8 KB of keys and values each.
  static constexpr int TS = RB >= 128 && !kBlocks ? 16 : 32;
  static constexpr int U = TS / 16;
  // What a unit costs beside its tiles (queries, merge, output: about 2 us of a
  // CTA), in tiles.  Without it, shares of many short rows finish last: 64 rows
  // up to 16384 tokens NVFP4 with 0, 1, 2, 3 tiles 116.8 us, 113.5, 109.3, 110.9;
  // 17 rows with a window, f16, with 1, 2, 3: 18.1, 17.6, 17.5.
  static constexpr int kLead = kQuant ? 2 : 3;
  static constexpr int kSide = TS * RB;          // keys, or values, of a step
  // The copies of a step: chunk i = kFill c + filler of a side is row i / CPR, bytes 16 (i % CPR)..;
  // both repeat every CY copies, CR rows further on.  The last copy may be for some warps only.
  static constexpr int CPR = RB / 16, kChunks = TS * CPR, kCopies = (kChunks + kFill - 1) / kFill;
  static constexpr int CY = CPR / gcd(kFill, CPR), CR = kFill * CY / CPR;
  static_assert(kChunks % 32 == 0 && (kCopies <= CY || (kCopies % CY == 0 && (CR & (CR - 1)) == 0)), "");
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
  static constexpr int kSlot = 2 * kSide + kRaw;
  // At a unit's end a warp hands its sums over in the slot that it read last,
  // kBox head tiles at a time.
  static constexpr int kBox = COLS > 1 ? NT : 2 * kSide / (MT * 4 * 32 * 4) < NT ? 2 * kSide / (MT * 4 * 32 * 4) : NT;
  // The queries of a block as operands: a head's row, 16 bytes apart from the next (bank conflicts).
  static constexpr int kQuery = DP * 2 + 16;
  static constexpr int kHeads = COLS * H;  // query heads of a block
  // Shared memory beside the rings.
  static constexpr int kRest = 128 + kWarps * kNotes + kWarps * (H * 8 + 8) + kHeads * (kQuery + 4);
  // Steps of a warp's ring with so many CTAs an SM.  More CTAs hide more
  // latency and keep the ALUs of 8- and 4-bit formats busier; the registers of
  // two head tiles or wide heads allow two or three.
  static constexpr int kMostSlots = COLS == 1 ? 6 : 10, kFewestSlots = COLS == 1 ? 2 : 4;
  static constexpr int slots(int ctas) {
    const int n = (kSmemSm / ctas - 1024 - kRest) / kRings / kSlot;
    return n < kMostSlots ? n : kMostSlots;
  }
  static constexpr int kMostCtas = (DP == 64 ? (NT == 1 ? 4 : 3) : DP * NT <= 128 ? 4 : 2) * 4 / kWarps;
  static constexpr int pick(int ctas) { return ctas == 1 || slots(ctas) >= kFewestSlots ? ctas : pick(ctas - 1); }
  static constexpr int kCtas = pick(kMostCtas);
  static constexpr int S = slots(kCtas);
  static constexpr int kRing = kRings * S * kSlot;
  static_assert(S >= kFewestSlots && 3 * S <= 32 && kBox >= 1 && NT % kBox == 0, "");
  static constexpr int kEarly = kHeads / kWarps < 4 ? kHeads / kWarps : 4;  // queries that a warp loads at a time
  // slots, notes and queries are read and written 16 bytes at a time
  static_assert(kSlot % 128 == 0 && kNotes % 16 == 0 && kWarps * (H * 8 + 8) % 16 == 0 && kQuery % 16 == 0, "");
};

// The place of a token among its step's (see the order of tokens above), and the token of a place.
__device__ __forceinline__ constexpr int place_of(int t) { return (t & ~7) + 2 * (t & 3) + ((t >> 2) & 1); }
__device__ __forceinline__ constexpr int token_at(int r) { return (r & ~7) + 4 * (r & 1) + ((r >> 1) & 3); }

// A warp's way through its CTA's share of the line, unit by unit.
struct Walk {
  int t, at, left;   // row, place in the row's line, numbers left in the share
  UnitPart part;     // what the share holds of the unit
  int seq;           // the row's sequence
  int first, base, stop;  // tokens: the first that counts, this warp's next step's, the end

  // The next unit of which the share holds tiles; false at the share's end.  A
  // row of a bad sequence has no steps.
  __device__ __forceinline__ bool next(const AttnArgs& a, int offset) {
    RowSpan s;
    do {
      if (left == 0) return false;
      s = span_of(a, t);
#pragma unroll 1
      while (at >= row_numbers(s.tiles, a.lead, a.units)) {
        at -= row_numbers(s.tiles, a.lead, a.units);
        s = span_of(a, ++t);
      }
      part = unit_part(at, left, s.tiles, a.lead);
      at += part.used;
      left -= part.used;
    } while (part.tiles == 0);
    seq = kv_seq(a.kv, t);
    first = s.first;
    base = s.begin + (part.tile0 << a.tile_log2) + offset;
    stop = min(s.len, s.begin + ((part.tile0 + part.tiles) << a.tile_log2));
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

  __device__ __forceinline__ void init(const AttnArgs& a, uint32_t ring, int column, int lane) {
#pragma unroll
    for (int c = 0; c < X::CY; ++c) {
      const int i = c * X::kFill + column * 32 + lane, row = i / X::CPR, chunk = i % X::CPR;
      src[0][c] = a.kv.data[0] + chunk * 16;
      src[1][c] = a.kv.data[1] + chunk * 16;
      kdst[c] = place_of(row) * X::RB + ((chunk * 16) ^ X::key_swizzle(place_of(row)));
      vdst[c] = X::kSide + row * X::RB + ((chunk * 16) ^ X::value_swizzle(row));
    }
    at = ring;
    past = 0;
  }

  // What stays the same over the walk's unit.  Its queries are fetched into L2
  // on the way: the reads of the cache that follow would hold them up.
  __device__ __forceinline__ void enter(const AttnArgs& a, int lane) {
    table = a.kv.pages + walk.seq * a.kv.table_stride;
    const int kv_head = walk.part.unit / a.blocks;
    head_row = static_cast<uint32_t>(kv_head) * a.kv.at.head_stride;
    const int h = (walk.part.unit - kv_head * a.blocks) * a.block_heads + lane;
    if (lane < a.block_heads && h < a.G) {
      const uint16_t* row = a.q + static_cast<int64_t>(walk.t) * a.q_tok + static_cast<int64_t>(kv_head * a.G + h) * a.q_head;
      asm volatile("prefetch.global.L2 [%0];" ::"l"(row));
      if (X::kQuery > 272) asm volatile("prefetch.global.L2 [%0];" ::"l"(row + (a.kv.D > 128 ? 128 : 0)));
    }
  }

  __device__ __forceinline__ void prepare(const AttnArgs& a, int offset, int step, int lane) {
    while (walk.base >= walk.stop) {
      if (!walk.next(a, offset)) {
        more = false;
        return;
      }
      enter(a, lane);
    }
    look_up(a, step, lane);
  }

  // The page of the lane's token of the step that the walk has come to.
  __device__ __forceinline__ void look_up(const AttnArgs& a, int step, int lane) {
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
        const uint32_t kb = held_exponent<X::kFmt>((kw >> sh) & 0xffu), vb = held_exponent<X::kFmt>((vw >> sh) & 0xffu);
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

  // Starts the prepared step's copies into its slot, which every thread of the
  // ring's warps has finished reading.  One group of copies a call, whether it
  // has any or not.
  __device__ __forceinline__ void issue(const AttnArgs& a, uint32_t ring, int column, int lane) {
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
          if (X::kCopies * X::kFill > X::kChunks && c * X::kFill + column * 32 >= X::kChunks) break;
          const int cy = c % X::CY, on = c / X::CY * X::CR;
          const uint32_t n = __shfl_sync(kAll, row, (cy * X::kFill + column * 32 + lane) / X::CPR + on);
          copy16(at + (kdst[cy] ^ X::key_swizzle(place_of(on))) + place_of(on) * X::RB,
                 src[0][cy] + static_cast<uint64_t>(n) * X::RB);
          copy16(at + (vdst[cy] ^ X::value_swizzle(on)) + on * X::RB, src[1][cy] + static_cast<uint64_t>(n) * X::RB);
        }
      } else {
#pragma unroll 1
        for (int i = column * 32 + lane; i < X::kChunks; i += X::kFill) {
          const int tok = i / X::CPR, chunk = i % X::CPR * 16;
          const uint32_t n = __shfl_sync(kAll, row, tok);
          const bool ok = n != kNoRow && chunk < a.kv.row_bytes;
          const uint64_t off = ok ? static_cast<uint64_t>(n) * a.kv.row_bytes + chunk : 0;
          const int pl = place_of(tok);
          copy16_or_zero(at + pl * X::RB + (chunk ^ X::key_swizzle(pl)), a.kv.data[0] + off, ok ? 16 : 0);
          copy16_or_zero(at + X::kSide + tok * X::RB + (chunk ^ X::value_swizzle(tok)), a.kv.data[1] + off, ok ? 16 : 0);
        }
      }
      if constexpr (X::kQuant) {
        if (has_row && column == 0) {
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

// The weights are rescaled when the greatest score exceeds the one that set the
// reference by this much (in powers of two), not at every new maximum.
constexpr float kSlack = 4.f;

template <typename X, int NT>
__device__ __forceinline__ void add_values(uint32_t at, uint32_t vnotes, int u, int g, int q,
                                           const uint32_t (&hi)[NT][2], const uint32_t (&lo)[NT][2],
                                           float (&acc)[X::MT][NT][4]) {
  const auto step = [&](int mt, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3) {
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      mma<X::kF16>(acc[mt][n], a0, a1, a2, a3, hi[n][0], hi[n][1]);
      mma<X::kF16>(acc[mt][n], a0, a1, a2, a3, lo[n][0], lo[n][1]);
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

// A row that sees nothing: zeros and -inf.
__device__ __noinline__ void empty_row(const AttnArgs& a, int t) {
  const bool f32 = a.out_f32 != 0;
#pragma unroll 1
  for (int i = threadIdx.x; i < a.Hq * (a.kv.D / 2); i += blockDim.x) {
    const int h = i / (a.kv.D / 2), d = 2 * (i - h * (a.kv.D / 2));
    const int64_t to = static_cast<int64_t>(t) * a.out_tok + static_cast<int64_t>(h) * a.out_head + d;
    if (f32)
      *reinterpret_cast<float2*>(static_cast<float*>(a.out) + to) = make_float2(0.f, 0.f);
    else
      *reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(a.out) + to) = 0;
    if (d == 0) store_lse(a, t, h, -INFINITY, 0.f);
  }
}

// Weights enter the value product as two 16-bit terms, so that an output is
// that of fp32 weights (3e-7 of the norm from the 64-bit one, as far as plain
// fp32 is).  With one f16 term each weight is up to 2^-11 off, and a few in a
// hundred of 16-bit outputs were rounded the other way (5e-4 of the norm); it took
// one row of 130999 E4M3 31.5 us and 64 rows up to 16384 NVFP4 99.8, the two terms
// 33.0 and 109.3.
template <int FMT, int DP, int NT, int COLS>
__global__ void __launch_bounds__(Deal<FMT, DP, NT, COLS>::kThreads, Deal<FMT, DP, NT, COLS>::kCtas)
    attend_kernel(const __grid_constant__ AttnArgs a) {
  using X = Deal<FMT, DP, NT, COLS>;
  constexpr int kWarps = X::kWarps, kWarpsT = X::kWarpsT;
  constexpr int U = X::U, MT = X::MT, H = X::H, S = X::S;
  extern __shared__ uint8_t smem_raw[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, q = lane & 3;
  const int wh = COLS > 1 ? warp : 0, wt = COLS > 1 ? 0 : warp;

  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 127) & ~uintptr_t(127));
  const uint32_t ring = smem_u32(smem) + wt * (S * X::kSlot);
  const uint32_t note = smem_u32(smem) + X::kRing + warp * X::kNotes;
  uint8_t* rest = smem + X::kRing + kWarps * X::kNotes;
  float2* sums = reinterpret_cast<float2*>(rest);                              // [warp][H] maximum and sum handed over
  uint32_t* box_of = reinterpret_cast<uint32_t*>(rest + kWarps * H * 8);         // [warp] where its accumulators are
  uint8_t* queries = rest + kWarps * (H * 8 + 8);                              // [head][kQuery]
  float* downs = reinterpret_cast<float*>(queries + X::kHeads * X::kQuery);  // [head] undoes the query's scaling

  pdl_wait();
  pdl_launch_dependents();

  // this CTA's share of the line, and the row it begins in
  Walk walk;
  {
    // rows that see nothing
#pragma unroll 1
    for (int t = blockIdx.x; t < a.T; t += gridDim.x)
      if (span_of(a, t).tiles == 0) empty_row(a, t);
    const Begin begin = begin_of<X::kThreads>(a, blockIdx.x);
    const int from = blockIdx.x * begin.share;
    if (from >= begin.total) return;
    walk.left = min(begin.share, begin.total - from);
    walk.t = begin.t;
    walk.at = begin.at;
  }
  walk.base = walk.stop = 0;
  const int offset = wt * X::TS, step = X::TS * kWarpsT;

  if (!walk.next(a, offset)) return;  // the share is the lead of a unit that begins in the next
  Feeder<X> feed;
  feed.walk = walk;
  feed.more = true;
  feed.enter(a, lane);
  // The first page is on its way while the rest is set up (777 tokens bf16 7.4 us
  // and 7.7).
  const bool early_page = walk.base < walk.stop;
  if (early_page) feed.look_up(a, step, lane);
  feed.init(a, ring, wh, lane);

  // places of the lane's pieces in a step's rows
  uint32_t koff[X::KP];
#pragma unroll
  for (int p = 0; p < X::KP; ++p) koff[p] = g * X::RB + ((p * 4 + q) * X::PK ^ X::key_swizzle(g));
  const uint32_t voff = q * X::RB + (g * X::PV ^ X::value_swizzle(q));

  // The queries of a unit, as loaded: the first unit's before the ring is
  // filled, for the same reason as in enter().
  int kv_head, head0;  // the key head, and the unit's first query head in its group
  const auto query = [&](int h) {
    uint4 raw = make_uint4(0, 0, 0, 0);
    if (head0 + h < a.G && lane * 8 < a.kv.D)
      raw = *reinterpret_cast<const uint4*>(a.q + static_cast<int64_t>(walk.t) * a.q_tok +
                                            static_cast<int64_t>(kv_head * a.G + head0 + h) * a.q_head + lane * 8);
    return raw;
  };
  uint4 early[X::kEarly];
  const auto enter = [&]() {
    kv_head = walk.part.unit / a.blocks;
    head0 = (walk.part.unit - kv_head * a.blocks) * a.block_heads;
#pragma unroll
    for (int i = 0; i < X::kEarly; ++i) early[i] = query(warp + i * kWarps);
  };
  enter();
#pragma unroll 1
  for (int i = 0; i < S; ++i) {
    if (i > 0) feed.issue(a, ring, wh, lane);
    if (feed.more && !(i == 0 && early_page)) feed.prepare(a, offset, step, lane);
  }

  uint32_t at = ring;  // the slot to read next
  uint32_t qb[MT][NT][2];
  float mul[NT][2], acc[MT][NT][4], m[NT][2], l[NT][2];
#pragma unroll 1
  while (true) {
    // Queries as B operands.  Where the products are f16, a head's row is
    // scaled by a power of two, undone in the scores' factor: its largest
    // element to [2^14, 2^15), so that bf16's eight bits are kept down to 2^31
    // below it (f16's steps end at 2^-24), and f16's eleven down to 2^28.
    const auto place = [&](int h, uint4 raw) {
      if (X::kF16) {
        float x[8];
        const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
        float amax = 0.f;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float2 v = a.q_f16 ? unpack16<true>(w[i]) : unpack16<false>(w[i]);
          x[2 * i] = v.x;
          x[2 * i + 1] = v.y;
          amax = fmaxf(amax, fmaxf(fabsf(v.x), fabsf(v.y)));
        }
        // positive floats order as their bits do
        amax = __uint_as_float(__reduce_max_sync(kAll, __float_as_uint(amax)));
        int e = 141 - static_cast<int>(__float_as_uint(amax) >> 23);
        e = amax > 0.f && amax <= 3.4028235e38f ? min(max(e, -120), 120) : 0;
        const float up = __uint_as_float((127 + e) << 23);
        raw = make_uint4(pack16<true>(x[0] * up, x[1] * up), pack16<true>(x[2] * up, x[3] * up),
                         pack16<true>(x[4] * up, x[5] * up), pack16<true>(x[6] * up, x[7] * up));
        if (lane == 0) downs[h] = __uint_as_float((127 - e) << 23);
      }
      if (lane * 8 < DP) *reinterpret_cast<uint4*>(queries + h * X::kQuery + lane * 16) = raw;
    };
#pragma unroll 1
    for (int h = warp; h < X::kHeads; h += X::kEarly * kWarps) {
      if (h > warp) {
#pragma unroll
        for (int i = 0; i < X::kEarly; ++i) early[i] = query(h + i * kWarps);
      }
#pragma unroll
      for (int i = 0; i < X::kEarly; ++i) place(h + i * kWarps, early[i]);
    }
    __syncthreads();
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const uint8_t* row = queries + (wh * H + n * 8 + g) * X::kQuery;
#pragma unroll
      for (int st = 0; st < MT; ++st) {
        constexpr int E = X::EK / 4;
        const uint2 b = *reinterpret_cast<const uint2*>(row + 2 * ((st / E) * 4 * X::EK + q * X::EK + (st % E) * 4));
        qb[st][n][0] = b.x;
        qb[st][n][1] = b.y;
      }
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        mul[n][i] = a.scale_log2 * (X::kF16 ? downs[wh * H + n * 8 + 2 * q + i] : 1.f);
        m[n][i] = kLowest;
        l[n][i] = 0.f;
      }
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[mt][n][i] = 0.f;
    }

    uint32_t last = 0;  // the slot that this unit's last step was read from; 0: none yet
#pragma unroll 1
    for (; walk.base < walk.stop; walk.base += step) {
      if (COLS > 1) {  // one barrier a step: its copies have landed, and the slot of the step before has been read
        asm volatile("cp.async.wait_group %0;" ::"n"(S - 2) : "memory");
        __syncthreads();
      } else {
        __syncwarp();
      }
      feed.issue(a, ring, wh, lane);  // fills the slot of the step before
      if (feed.more) feed.prepare(a, offset, step, lane);
      if (COLS == 1) {
        asm volatile("cp.async.wait_group %0;" ::"n"(S - 1) : "memory");
        __syncwarp();
      }
      feed.put_notes(at, note, lane);

      // s[u][n] = S^T of 16 tokens: (token g | g + 8) x (head 2q | 2q + 1)
      float s[U][NT][4];
#pragma unroll
      for (int u = 0; u < U; ++u) {
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int i = 0; i < 4; ++i) s[u][n][i] = 0.f;
        constexpr bool kTwoSums = U == 1;
        float s2[NT][4] = {};
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
              mma<X::kF16>(kTwoSums && (i & 1) ? s2[n] : s[u][n], f[0][2 * i], f[1][2 * i], f[0][2 * i + 1], f[1][2 * i + 1],
                           qb[st][n][0], qb[st][n][1]);
            }
        }
        if (kTwoSums) {
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i) s[u][n][i] += s2[n][i];
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
              // the key's exponent last: q.k of codes stays in range, and so does every finite score
              x = X::kQuant ? fmaf(x * mul[n][i], ks, ev) : x * mul[n][i];
              if (part) x = ok ? x : -INFINITY;
              more |= x > m[n][i] + (kSlack + X::kLift);
            }
        }
      if (__any_sync(kAll, more)) {
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            float top = -INFINITY;
#pragma unroll
            for (int u = 0; u < U; ++u) top = fmaxf(top, fmaxf(s[u][n][i], s[u][n][2 + i]));
            top = fmaxf(top, __shfl_xor_sync(kAll, top, 4));
            top = fmaxf(top, __shfl_xor_sync(kAll, top, 8));
            top = fmaxf(top, __shfl_xor_sync(kAll, top, 16));
            top = fmaxf(m[n][i], top - X::kLift);
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
            const float2 back = unpack16<X::kF16>(h);
            lo[n][r] = transpose8x8(pack16<X::kF16>(p0 - back.x, p1 - back.y));
          }
        }
        const uint32_t vnotes = note + X::kTok + X::kKeyBlk;
        add_values<X, NT>(at + X::kSide + voff, vnotes, u, g, q, hi, lo, acc);
      }

      last = at;
      at += X::kSlot;
      if (at == ring + S * X::kSlot) at = ring;
    }

    // The next unit's queries are requested before this one is handed over.
    const int t = walk.t, hq0 = kv_head * a.G + head0, heads = min(a.block_heads, a.G - head0);
    const UnitPart unit = walk.part;
    const bool more = walk.next(a, offset);
    if (more) enter();

    // The unit's end.  A lane has of two heads (8n + 2q, + 1) and 16 channels a
    // mt the four sums c: (channel d, d + 1) x (head, head + 1).
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        l[n][i] += __shfl_xor_sync(kAll, l[n][i], 4);
        l[n][i] += __shfl_xor_sync(kAll, l[n][i], 8);
        l[n][i] += __shfl_xor_sync(kAll, l[n][i], 16);
      }
    const bool whole = unit.rest == 0 && unit.tile0 == 0;
    const int part = blockIdx.x * 2 + (unit.tile0 == 0 ? 1 : 0);
    const bool f32 = !whole || a.out_f32 != 0;
    const int64_t on = whole ? a.out_head : DP;  // to the next head
    const auto place_of_head = [&](int h) {
      return whole ? static_cast<int64_t>(t) * a.out_tok + static_cast<int64_t>(hq0 + h) * a.out_head
                   : (static_cast<int64_t>(part) * X::kHeads + h) * DP;
    };
    const auto norm_of = [&](float L) { return !whole ? 1.f : L == 0.f ? 0.f : 1.f / L; };
    // maxima and sums of the heads h and h + 1
    const auto write_sums = [&](int h, const float (&M)[2], const float (&L)[2]) {
      if (g < 2 && wt == 0 && h + g < heads) {
        const float mg = g ? M[1] : M[0], lg = g ? L[1] : L[0];
        if (whole)
          store_lse(a, t, hq0 + h + g, mg, lg);
        else
          a.part_ml[part * X::kHeads + h + g] = make_float2(mg, lg);
      }
    };
    const auto write = [&](int h, int64_t to, int mt, const float (&c)[4], const float (&norm)[2]) {
      const int d = (mt / (X::EV / 2)) * 8 * X::EV + g * X::EV + 2 * (mt % (X::EV / 2));
      if (whole && d >= a.kv.D) return;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        if (h + i >= heads) continue;
        const int64_t at_d = to + i * on + d;
        float x = c[i] * norm[i], y = c[2 + i] * norm[i];
        if (!X::kQuant && whole) x = finite_or_nan(x), y = finite_or_nan(y);
        if (f32)
          *reinterpret_cast<float2*>((whole ? static_cast<float*>(a.out) : a.part_o) + at_d) = make_float2(x, y);
        else
          *reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(a.out) + at_d) = pack_out(a, x, y);
      }
    };
    if constexpr (COLS > 1) {  // a warp has its heads' sums
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        const int h = wh * H + n * 8 + 2 * q;  // in the block
        const float norm[2] = {norm_of(l[n][0]), norm_of(l[n][1])};
        const int64_t to = place_of_head(h);
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) write(h, to, mt, acc[mt][n], norm);
        write_sums(h, m[n], l[n]);
      }
    } else {
      // The warps' sums meet in shared memory, and each warp joins and writes a
      // part of the channels.  A warp with steps has read a slot, which is not
      // filled again before the next unit.  One without has nothing to add; then
      // warps after it have no steps either, and its sums are those of nothing.
#pragma unroll
      for (int n = 0; n < NT; ++n)
        if (g < 2) sums[warp * H + n * 8 + 2 * q + g] = make_float2(g ? m[n][1] : m[n][0], g ? l[n][1] : l[n][0]);
      if (lane == 0) box_of[warp] = last;
#pragma unroll
      for (int n0 = 0; n0 < NT; n0 += X::kBox) {
        if (n0 > 0) __syncthreads();  // the tiles before have been read
        if (last != 0) {
#pragma unroll
          for (int n = n0; n < n0 + X::kBox; ++n)
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
              asm volatile("st.shared.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(last + ((n - n0) * MT + mt) * 512 + lane * 16),
                           "f"(acc[mt][n][0]), "f"(acc[mt][n][1]), "f"(acc[mt][n][2]), "f"(acc[mt][n][3])
                           : "memory");
        }
        __syncthreads();
        // where the warps' sums are; the first's in the place of one that has
        // none (whose weight is 0); where none has any, the ring's start is read
        // and not used
        const uint32_t first = box_of[0], other = first != 0 ? first : smem_u32(smem);
        uint32_t box[kWarps];
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
          const uint32_t own = box_of[w];
          box[w] = (own != 0 ? own : other) + lane * 16;
        }
#pragma unroll
        for (int n = n0; n < n0 + X::kBox; ++n) {
          // the warps' weights for the heads 2q and 2q + 1
          float M[2], L[2], y[kWarps][2], norm[2];
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            float2 o[kWarps];
            M[i] = kLowest;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
              o[w] = sums[w * H + n * 8 + 2 * q + i];
              M[i] = fmaxf(M[i], o[w].x);
            }
            L[i] = 0.f;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
              y[w][i] = weight_of(o[w].x, M[i]);
              L[i] = fmaf(o[w].y, y[w][i], L[i]);
            }
          }
          norm[0] = norm_of(L[0]);
          norm[1] = norm_of(L[1]);
          // The sums of all the warp's tiles are read at once: one wait for shared
          // memory (NVFP4, whose registers are short: of one tile at a time).
          constexpr int kTiles = X::kBlocks ? 1 : MT / kWarps;
          const int h = n * 8 + 2 * q;  // in the block
          const int64_t to = place_of_head(h);
#pragma unroll 1
          for (int mt = wt; mt < MT; mt += kTiles * kWarps) {
            float o[kTiles][kWarps][4];
#pragma unroll
            for (int j = 0; j < kTiles; ++j)
#pragma unroll
              for (int w = 0; w < kWarps; ++w)
                asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];"
                             : "=f"(o[j][w][0]), "=f"(o[j][w][1]), "=f"(o[j][w][2]), "=f"(o[j][w][3])
                             : "r"(box[w] + ((n - n0) * MT + mt + j * kWarps) * 512));
#pragma unroll
            for (int j = 0; j < kTiles; ++j) {
              float c[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
              for (int w = 0; w < kWarps; ++w)
#pragma unroll
                for (int i = 0; i < 4; ++i) c[i] = fmaf(o[j][w][i], y[w][i & 1], c[i]);
#pragma unroll
              for (int i = 0; i < 4; ++i) c[i] = first != 0 ? c[i] : 0.f;
              write(h, to, mt + j * kWarps, c, norm);
            }
          }
          write_sums(h, M, L);
        }
      }
    }
    if (!more) break;
    __syncthreads();  // the unit has been handed over: its slots and queries are free
  }
}

// ------------------------------------------------------------------ host side ---
template <int FMT, int DP, int NT, int COLS>
ft_status launch(AttnArgs& a, cudaStream_t s) {
  using X = Deal<FMT, DP, NT, COLS>;
  const auto kernel = attend_kernel<FMT, DP, NT, COLS>;
  constexpr int smem = X::kRing + X::kRest;
  ft_status st = ensure_dyn_smem(reinterpret_cast<const void*>(kernel), smem, "attn_decode");
  if (st != FT_OK) return st;
  static std::atomic<int> held{0};  // CTAs an SM holds
  int r = held.load(std::memory_order_relaxed);
  if (r == 0) {
    if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&r, kernel, X::kThreads, smem) != cudaSuccess || r < 1)
      return fail(FT_ERR_CUDA, "attn_decode: %s", cudaGetErrorString(cudaGetLastError()));
    held.store(r, std::memory_order_relaxed);
  }
  constexpr int tile = X::TS * X::kWarpsT;
  a.tile_log2 = log2_of(tile);
  a.lead = X::kLead;
  a.lift = X::kLift;
  const int32_t longest = a.window > 0 && a.window < a.most - 15 ? a.window + 15 : a.most;
  const int64_t most_tiles = (int64_t{row_span(longest, 0, longest, tile).tiles} + a.lead) * a.units * a.T;
  // the line's numbers are 32-bit in the kernel
  if (most_tiles >= (1ll << 31) - kMaxWorkers) return fail(FT_ERR_UNSUPPORTED, "attn_decode: rows times pages too large");
  int64_t workers = static_cast<int64_t>(device_sm_count()) * r;
  if (workers > kMaxWorkers) workers = kMaxWorkers;
  if (workers > most_tiles) workers = most_tiles;
  a.workers = static_cast<int>(workers);
  return launch_pdl(kernel, dim3(a.workers), X::kThreads, smem, s, a, "attn_decode");
}

template <int FMT, int DP, int NT>
ft_status launch_columns(AttnArgs& a, const AttnShape& sh, cudaStream_t s) {
  if (sh.columns == 4) return launch<FMT, DP, NT, 4>(a, s);
  if (sh.columns == 2) return launch<FMT, DP, NT, 2>(a, s);
  return launch<FMT, DP, NT, 1>(a, s);
}

template <int FMT>
ft_status launch_shape(AttnArgs& a, const AttnShape& sh, cudaStream_t s) {
  switch (sh.DP) {
    case 64: return sh.NT == 2 ? launch_columns<FMT, 64, 2>(a, sh, s) : launch<FMT, 64, 1, 1>(a, s);
    case 128: return sh.NT == 2 ? launch_columns<FMT, 128, 2>(a, sh, s) : launch<FMT, 128, 1, 1>(a, s);
    case 192: return launch_columns<FMT, 192, 1>(a, sh, s);
    default: return launch_columns<FMT, 256, 1>(a, sh, s);
  }
}

}  // namespace
}  // namespace ft
