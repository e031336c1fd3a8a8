// ft_attn_args.cuh -- what attn.cu and the attention kernels share: the
// arguments, the shapes, and the launch of each format's kernel.
#pragma once

#include "ft_kv.cuh"

namespace ft {

constexpr int kMaxWorkers = 1024;  // CTAs of one call (sizes the workspace)

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
  int32_t block_heads;   // heads of a block
  int32_t tile_log2;     // tokens of a CTA's tile: a power of two, because kernels divide by them in many places
  int32_t lead;          // numbers of a unit in the line before those of its tiles
  int32_t most;          // max_pages * page_size
  int32_t q_f16, out_f32;
  int32_t workers;
  int32_t lift;          // weights' reference lies this many powers of two below the greatest score
  int32_t* status;
};

__device__ __forceinline__ RowSpan span_of(const AttnArgs& a, int t) {
  return row_span_log2(a.lens[t], a.window, a.most, a.tile_log2);
}

__device__ __forceinline__ int numbers_of(const AttnArgs& a, int t) {
  return row_numbers(span_of(a, t).tiles, a.lead, a.units);
}

// Where worker `c`'s share begins: the share's size, the line's length, and
// (where the share begins inside the line) the row and the place in its
// numbers.  By the whole block; every thread must call it.
struct Begin {
  int share, total;
  int t, at;
};

template <int kThreads>
__device__ __forceinline__ Begin begin_of(const AttnArgs& a, int c) {
  Begin r;
  const int lane = threadIdx.x & 31;
  if (a.T <= 32) {  // every warp for itself, a row a lane
    const int n = lane < a.T ? numbers_of(a, lane) : 0;
    int upto = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, upto, o);
      if (lane >= o) upto += y;
    }
    r.total = __shfl_sync(0xffffffffu, upto, 31);
    r.share = split_share(r.total, a.workers);
    const int from = c * r.share;
    r.t = max(__ffs(__ballot_sync(0xffffffffu, upto > from)) - 1, 0);
    r.at = from - __shfl_sync(0xffffffffu, upto - n, r.t);
  } else {  // neighbouring rows a thread: 1024 rows by every warp for itself took 40 us more
    __shared__ int scratch[33];
    __shared__ int2 begin;
    const int each = (a.T + kThreads - 1) / kThreads, first = threadIdx.x * each;
    int own = 0;
#pragma unroll 1
    for (int t = first; t < min(first + each, a.T); ++t) own += numbers_of(a, t);
    int before = block_excl_scan(own, scratch, &r.total);
    r.share = split_share(r.total, a.workers);
    const int from = c * r.share;
    if (before <= from && from < before + own) {
      int t = first;
#pragma unroll 1
      for (int n = numbers_of(a, t); before + n <= from; n = numbers_of(a, ++t)) before += n;
      begin = make_int2(t, from - before);
    }
    __syncthreads();
    r.t = begin.x;
    r.at = begin.y;
  }
  return r;
}

// Softmax weights are taken in powers of two, 2^(x - m), with a reference m
// that is `lift` below (about) the greatest score, above it where negative.  A
// maximum over nothing is kLowest: finite, so that 2^(-inf - kLowest) and
// 2^(kLowest - m) are 0 and not NaN.
constexpr float kLowest = -3.4028235e38f;  // the lowest fp32

__device__ __forceinline__ float exp2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float weight_of(float m, float M) { return exp2_approx(m - M); }

// The logarithm of a head's sum l of weights with the reference m.  The lift is
// taken off both: exactly, and without it log2(l) and m cancel to fewer bits.
__device__ __forceinline__ void store_lse(const AttnArgs& a, int t, int h, float m, float l) {
  if (a.lse == nullptr) return;
  const float sum = l * __uint_as_float((127 - a.lift) << 23);
  a.lse[static_cast<int64_t>(t) * a.Hq + h] =
      l > 0.f || l != l ? (m + static_cast<float>(a.lift) + log2f(sum)) * 0.69314718055994531f : -INFINITY;
}

// An output of a 16-bit cache.  Its weighted mean is finite unless a value that
// counts is not, and with an infinity the two terms of a weight, or a weight
// that rounds to 0, may give an infinity or NaN: it is NaN throughout.
__device__ __forceinline__ float finite_or_nan(float x) { return __fmaf_rn(x, 0.f, x); }

// Two output values in one word.
__device__ __forceinline__ uint32_t pack_out(const AttnArgs& a, float x, float y) {
  uint32_t d;
  if (a.q_f16)
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(y), "f"(x));
  else
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(y), "f"(x));
  return d;
}

struct AttnShape {
  int DP, NT;        // channels padded to 64s; 8-head column tiles of a warp
  int columns, block_heads, blocks;  // warps side by side over a block's heads
};

// The kernel of each cache format; sets a.tile_log2, a.lead, a.lift and a.workers.
ft_status attend_bf16(AttnArgs& a, const AttnShape& sh, cudaStream_t s);
ft_status attend_f16(AttnArgs& a, const AttnShape& sh, cudaStream_t s);
ft_status attend_e4m3(AttnArgs& a, const AttnShape& sh, cudaStream_t s);
ft_status attend_nvfp4(AttnArgs& a, const AttnShape& sh, cudaStream_t s);

}  // namespace ft
