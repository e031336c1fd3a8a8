// ft_fp4_matmul.cuh -- the product of two microscaled 4-bit matrices, X [T, K] and
// W [N, K], on the block-scaled tensor cores.
//
// A tile is 128 rows of W (the M side, TMEM's lanes), or 256 over a pair of CTAs,
// by up to 256 tokens (the N side, its columns): one token's product then costs no
// more than the weights' bytes.  A step is 256 values of K: 128 bytes of codes a
// row, by TMA in the 128-byte swizzle, and the scale tiles (512 bytes for 128 rows x
// 4 scales) as they lie in memory, copied from shared memory to TMEM by the thread
// that issues the products, in front of them.  Each stage of the ring has scale
// columns of its own, so that a stage's release covers them.
//
// One warp issues the copies, one the products, eight drain the sums: where out is
// written by boxes, all of a tile's at once into registers, so that the next tile's
// products can begin; tiles of at most 128 tokens have two accumulators besides.  A CTA, or a pair, walks
// tiles; where there are few, K is cut into slices over the CTAs of a cluster, whose
// partial sums meet through distributed shared memory and are added in the slices'
// order.
//
// What bounds it.  64 x 131072 x 2048 reads its weights at 5.4 TB/s (28.2 us; floor
// 24.8).  8192 x 6144 x 4096 takes 73.5 us, 5.6 PFLOP/s, 8192^3 160, 6.9: a step of a
// 256 x 256 pair takes 0.30 us where its products alone take 0.27 (9.4 PFLOP/s), the
// copies of scales to TMEM 0.02 more and contention in shared memory the rest
// (operands are read at 64 bytes a clock, filled at 75); each tile adds 1 us in which
// its sums are drained; 768 tiles on 76 pairs are 10.1 waves.  Narrower tiles are bound
// by issuing: a step takes 0.255 us at 64 tokens, of which its barrier 0.15.  Calls of
// a few tokens, 4.7 us for 1 x 2560 x 2048, are launch, first loads and the way out.
// Rows of out off 16-byte boundaries are bound by their way out, which stands still
// for the products of tiles of more than 128 tokens: 8000 x 9998 x 1024 69 us (floor
// 25), 8000 x 9999 x 1024 onto a residual 149 (49); fp32 likewise, 2048 x 4096 x 4096
// 21.8 us (7.0).
//
// Tried and not kept: the next step's scales copied to TMEM ahead of this step's
// products (8192 x 6144 x 4096: 87.5 us, then 75.1); scale copies between the
// products that need them (no change); asking for the next step's barrier while a
// step is issued (75.2, then 76.0); the first steps' copies before the CTA has met
// (1 x 2560 x 2048: 5.5, then 5.5).
#pragma once

#include <algorithm>

#include "ft_fp4_args.cuh"
#include "ft_narrow.cuh"
#include "ft_tensor.cuh"

namespace ft {
namespace {

template <int DT>
__device__ __forceinline__ float load_out(const void* p, int64_t at) {
  if (DT == FT_DT_F32) return static_cast<const float*>(p)[at];
  return load_one<DT == FT_DT_F16>(static_cast<const uint16_t*>(p) + at);
}

template <int DT>
__device__ __forceinline__ void store_out(void* p, int64_t at, float x) {
  if (DT == FT_DT_F32)
    static_cast<float*>(p)[at] = x;
  else if (DT == FT_DT_F16)
    static_cast<__half*>(p)[at] = __float2half_rn(x);
  else
    static_cast<__nv_bfloat16*>(p)[at] = __float2bfloat16_rn(x);
}

// Where a tile lies: its tile of weight rows, its first token, how many it has.
struct Place {
  int w, t0, tokens;
};
__device__ __forceinline__ Place place_of(const MmArgs& a, int tile) {
  const int outer = tile / a.inner, in = tile - outer * a.inner;
  Place p;
  p.w = a.x_inner ? outer : in;
  p.t0 = (a.x_inner ? in : outer) * a.width;
  p.tokens = min(a.width, a.T - p.t0);
  return p;
}

// Columns of a product over these tokens: whole 16s of each CTA's.
template <int CG>
__device__ __forceinline__ int columns_of(int tokens) { return (tokens + 16 * CG - 1) & ~(16 * CG - 1); }

// A chunk of sums, 32 rows (TMEM lanes) x 32 tokens, as a warp's lanes hold it:
// value i is of row row_of(i) and token token(i).
struct Fragment {
  int row, col;               // of value 0
  int box_token, box_chunk;   // the lane's row of four 8 x 8 matrices in a box, and its 16-byte place there
  __device__ __forceinline__ int row_of(int i) const { return row + (i >> 4) * 16 + (i >> 1 & 1) * 8; }
  __device__ __forceinline__ int token(int i) const { return (i >> 2 & 3) * 8 + col + (i & 1); }
};
__device__ __forceinline__ Fragment fragment_of(int lane) {
  return Fragment{lane >> 2, 2 * (lane & 3), (lane >> 4) * 8 + (lane & 7), (lane >> 3) & 1};
}

// Its loads, in flight until tmem_wait.
__device__ __forceinline__ void tmem_ld32x32(uint32_t from, uint32_t (&v)[32]) {
  tmem_ld16x32(from, v);
  tmem_ld16x32(from + (16u << 16), v + 16);
}

// The 8 values of 16 tokens (from 8 k) x 16 rows (from 16 half), scaled.
__device__ __forceinline__ void scaled(const uint32_t (&v)[32], const float (&sw)[4], const float (&s)[4], int k, int half,
                                       float (&y)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i)
    y[i] = __uint_as_float(v[16 * half + 4 * k + i]) * sw[2 * half + (i >> 1 & 1)] * s[2 * (i >> 2) + (i & 1)];
}
__device__ __forceinline__ void scales_of(float sx_of_lane, const Fragment& f, int k, float (&s)[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) s[i] = __shfl_sync(0xffffffffu, sx_of_lane, (k + (i >> 1)) * 8 + f.col + (i & 1));
}

// Sums are 0 or 2^-20 to 2^54 in size.  By a weight row's scale of 2^-100 to 2^71 (or
// 0) they are neither infinite nor below the normal numbers, and sum * row's *
// token's is rounded as the whole.  Other scales are `far`: taken as near * by, near
// in that range and by a power of two that leads further the same way, so that ((sum
// * near) * token's) * by is rounded as the whole.
__device__ __forceinline__ bool far_scale(float s) {
  const uint32_t m = __float_as_uint(s) & 0x7fffffffu;  // magnitudes order as their bits do
  return m - 1 < (27u << 23) - 1 || m - (198u << 23) < (57u << 23);
}
struct RowScale {
  float near, by;
};
__device__ __forceinline__ RowScale split_scale(float s) {
  RowScale r = {s, 1.f};
  if (far_scale(s)) {
    const bool small = fabsf(s) < 1.f;
    const float t = small ? s * 0x1p49f : s;  // a normal number
    const int e = static_cast<int>(__float_as_uint(t) >> 23 & 255) - 127, to = small ? -100 : 70;
    r.near = __uint_as_float(__float_as_uint(t) + (static_cast<uint32_t>(to - e) << 23));
    r.by = pow2f(e - (small ? 49 : 0) - to);
  }
  return r;
}

// A warp's sums of a tile, `chunks` of every other 32 columns from `from`, scaled
// where they are: what follows then scales by 1.  In few registers and off the way of
// the tiles without far scales, which are nearly all (8000 x 9999 x 1024 takes 74.1 us
// without far scales, 77.8 so, 89 with a third factor for every value; asked for with
// the tile's own scales, not a tile ahead, 85.9).
__device__ __forceinline__ void scale_in_tmem(uint32_t from, int chunks, const float (&sw)[4], const float* sx,
                                              int64_t sx_stride, int tokens, const Fragment& f) {
#pragma unroll 1
  for (int j = 0; j < 8 * chunks; ++j) {
    const int half = j >> 2 & 1, column = (j >> 3) * 64 + (j & 3) * 8;
    const uint32_t at = from + column + (static_cast<uint32_t>(half * 16) << 16);
    uint32_t v[4];
    tmem_ld16x8(at, v);
    tmem_wait();
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int t = column + f.col + (i & 1);
      const RowScale w = split_scale(half != 0 ? sw[2 + (i >> 1)] : sw[i >> 1]);
      const float x = sx != nullptr && t < tokens ? sx[t * sx_stride] : 1.f;
      v[i] = __float_as_uint(__uint_as_float(v[i]) * w.near * x * w.by);
    }
    tmem_st16x8(at, v);
  }
  tmem_wait_stores();
}

// A warp's 32 tokens x 32 rows of 16-bit outputs in shared memory: 64 bytes a
// token, in the 64-byte swizzle.
__device__ __forceinline__ uint32_t box_at(uint32_t box, int token, int chunk) {
  return box + token * 64 + ((chunk ^ ((token >> 1) & 3)) << 4);
}

// A chunk scaled, rounded and put into a box, which holds what is added to it before.
template <int DT>
__device__ __forceinline__ void chunk_to_box(const uint32_t (&v)[32], const float (&sw)[4], float sx_of_lane,
                                             const Fragment& f, uint32_t box, bool added) {
#pragma unroll
  for (int k = 0; k < 4; k += 2) {
    float s[4];
    scales_of(sx_of_lane, f, k, s);
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      float y[8];
      scaled(v, sw, s, k, half, y);
      const uint32_t at = box_at(box, k * 8 + f.box_token, 2 * half + f.box_chunk);
      uint32_t r[4];
      if (added) {
        load_transposed(at, r);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float2 m = unpack2<DT == FT_DT_F16>(r[i]);
          y[2 * i] += m.x;
          y[2 * i + 1] += m.y;
        }
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) r[i] = pack2<DT == FT_DT_F16>(y[2 * i], y[2 * i + 1]);
      store_transposed(at, r);
    }
  }
}

// What is added to a chunk, on its way: fp32 as the sums lie; 16-bit rows a
// token's 32 over the lanes, or (`words`) two tokens', two rows a lane.  Past the last token or row it is the last one again: branches would have
// each load wait for the one before (1237 x 5003 x 2592: 44.7 us so).
template <int DT>
struct Added {
  uint32_t x[32];
};
template <int DT>
__device__ __forceinline__ void load_added(const MmArgs& a, int t, int n, const Fragment& f, Added<DT>& to) {
  const int lane = threadIdx.x & 31;
  const auto at = [&](int token, int row) { return static_cast<int64_t>(min(token, a.T - 1)) * a.add_stride + row; };
  if constexpr (DT == FT_DT_F32) {
#pragma unroll
    for (int i = 0; i < 32; ++i) to.x[i] = static_cast<const uint32_t*>(a.add)[at(t + f.token(i), min(n + f.row_of(i), a.N - 1))];
  } else if (a.words) {
    const int i = lane >> 4, m = min(n + 2 * (lane & 15), a.N - 2);
#pragma unroll
    for (int j = 0; j < 16; ++j)
      to.x[j] = *reinterpret_cast<const uint32_t*>(static_cast<const uint16_t*>(a.add) + at(t + 2 * j + i, m));
  } else {
    const int m = min(n + lane, a.N - 1);
#pragma unroll
    for (int j = 0; j < 32; ++j) to.x[j] = static_cast<const uint16_t*>(a.add)[at(t + j, m)];
  }
}

// 16-bit rows from there into the warp's box.
__device__ __forceinline__ void added_to_box(const MmArgs& a, const uint32_t (&x)[32], uint32_t box) {
  const int lane = threadIdx.x & 31;
  if (a.words) {
#pragma unroll
    for (int j = 0; j < 16; ++j) st_shared_u32(box_at(box, 2 * j + (lane >> 4), (lane & 15) >> 2) + (lane & 3) * 4, x[j]);
  } else {
#pragma unroll
    for (int j = 0; j < 32; ++j)
      st_shared_u16(box_at(box, j, lane >> 3) + (lane & 7) * 2, static_cast<uint16_t>(x[j]));
  }
  __syncwarp();
}

// A chunk scaled, added to and written where rows are not on 16-byte boundaries:
// through the warp's box, so that a store is of one token's 32 rows, or (`words`)
// of two tokens', two rows a lane.  fp32: as the sums lie, 8 rows of 4 tokens a
// store.  WHOLE: nothing of it is past the last row or token, so that stores need
// no branches.
template <int DT, bool WHOLE>
__device__ __forceinline__ void chunk_to_rows(const MmArgs& a, const uint32_t (&v)[32], const float (&sw)[4], float sx_of_lane,
                                              const Fragment& f, int t, int n, const Added<DT>& add, uint32_t box) {
  const int lane = threadIdx.x & 31;
  if constexpr (DT != FT_DT_F32) {
    if (a.add != nullptr) added_to_box(a, add.x, box);
    chunk_to_box<DT>(v, sw, sx_of_lane, f, box, a.add != nullptr);
  } else {
#pragma unroll
    for (int k = 0; k < 4; k += 2) {
      float s[4];
      scales_of(sx_of_lane, f, k, s);
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        float y[8];
        scaled(v, sw, s, k, half, y);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const int i = 16 * half + 4 * k + j;
          if (a.add != nullptr) y[j] += __uint_as_float(add.x[i]);
          if (WHOLE || (t + f.token(i) < a.T && n + f.row_of(i) < a.N))
            store_out<DT>(a.out, (t + f.token(i)) * a.out_stride + n + f.row_of(i), y[j]);
        }
      }
    }
  }
  if constexpr (DT != FT_DT_F32) {
    __syncwarp();
    if (a.words) {
      const int i = lane >> 4, m = n + 2 * (lane & 15);
      uint16_t* const to = static_cast<uint16_t*>(a.out) + (t + i) * a.out_stride + m;
      uint32_t x[16];
#pragma unroll
      for (int j = 0; j < 16; ++j) x[j] = ld_shared_u32(box_at(box, 2 * j + i, (lane & 15) >> 2) + (lane & 3) * 4);
#pragma unroll
      for (int j = 0; j < 16; ++j)
        if (WHOLE || (t + 2 * j + i < a.T && m < a.N)) *reinterpret_cast<uint32_t*>(to + 2 * j * a.out_stride) = x[j];
    } else {
      uint16_t* const to = static_cast<uint16_t*>(a.out) + t * a.out_stride + n + lane;
      uint16_t x[32];
#pragma unroll
      for (int j = 0; j < 32; ++j) x[j] = ld_shared_u16(box_at(box, j, lane >> 3) + (lane & 7) * 2);
#pragma unroll
      for (int j = 0; j < 32; ++j)
        if (WHOLE || (t + j < a.T && n + lane < a.N)) to[j * a.out_stride] = x[j];
    }
    __syncwarp();
  }
}

// BOXES: 16-bit rows of out (and add) on 16-byte boundaries, moved by whole boxes.
template <int FMT, int DT, int CG, bool BOXES>
__global__ void __launch_bounds__(kThreads, 1) matmul_kernel(const __grid_constant__ Maps maps,
                                                             const __grid_constant__ MmArgs a) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* const smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  __shared__ __align__(8) uint64_t full[kMaxStages], empty[kMaxStages], acc_full[2], acc_empty[2];
  __shared__ uint32_t s_tmem;
  __shared__ int s_bad, s_skip;
  __shared__ __align__(8) uint64_t add_full[kEpilogueWarps];
  uint32_t add_phase = 0;
  constexpr int kTiles = step_tiles<FMT>();
  constexpr int kRows = kM * CG;  // weight rows of a tile
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const int rank = CG == 2 || a.split > 1 ? static_cast<int>(cluster_rank()) : 0;
  const int slice = CG == 2 ? 0 : rank;
  const int s0 = static_cast<int>(static_cast<int64_t>(a.steps) * slice / a.split);
  const int s1 = static_cast<int>(static_cast<int64_t>(a.steps) * (slice + 1) / a.split);
  const int first = blockIdx.x / (CG * a.split), stride = gridDim.x / (CG * a.split);
  const int x_rows = a.width / CG;  // tokens that a CTA loads of a tile
  const int x_at = kM * 128, scales_at = x_at + x_rows * 128;
  constexpr int kWScales = kTiles * 512;

  if (threadIdx.x == 0) {
    prefetch_map(&maps.w);
    prefetch_map(&maps.x);
    prefetch_map(&maps.w_scales);
    prefetch_map(&maps.x_scales);
    if (BOXES) prefetch_map(&maps.out);
    for (int i = 0; i < a.stages; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&acc_full[i], 1);
      mbar_init(&acc_empty[i], kEpilogueWarps * CG);
    }
    for (int i = 0; i < kEpilogueWarps; ++i) mbar_init(&add_full[i], 1);
    s_bad = s_skip = 0;
    fence_barrier_init();
  }
  if (warp == 1) tmem_alloc<CG>(&s_tmem, 512);
  tc_fence_before();
  if (CG == 2) cluster_sync();
  else __syncthreads();
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, s_tmem, 0);
  pdl_wait();
  if (a.T <= kFewRows) pdl_launch_dependents();
  if (warp == 0) {
    int st = 0;
    uint32_t ph = 1;
    bool ok = true;
    const uint32_t bytes = CG * (kM * 128 + x_rows * 128 + kWScales * (1 + a.x_tiles));
    for (int tile = first; tile < a.tiles && ok; tile += stride) {
      const Place p = place_of(a, tile);
      const int n0 = p.w * kRows + (CG == 2 ? rank * kM : 0);
      const int x0 = p.t0 + (CG == 2 ? rank * (columns_of<CG>(p.tokens) / 2) : 0);
      for (int s = s0; s < s1; ++s) {
        if (!mbar_wait_warp<true>(&empty[st], ph, a.status)) {
          ok = false;
          break;
        }
        if (elect_one()) {
          uint8_t* const at = smem + st * a.stage_bytes;
          if (CG == 2) {
            const uint32_t bar = map_cluster(smem_u32(&full[st]), 0);
            if (rank == 0) mbar_arrive_expect_tx(&full[st], bytes);
            tma_load_2d_pair(at, &maps.w, s * 128, n0, bar);
            tma_load_2d_pair(at + x_at, &maps.x, s * 128, x0, bar);
            tma_load_2d_pair(at + scales_at, &maps.w_scales, s * kTiles * 64, n0 / 128, bar);
            tma_load_2d_pair(at + scales_at + kWScales, &maps.x_scales, s * kTiles * 64, p.t0 / 128, bar);
          } else {
            mbar_arrive_expect_tx(&full[st], bytes);
            tma_load_2d(at, &maps.w, s * 128, n0, &full[st]);
            tma_load_2d(at + x_at, &maps.x, s * 128, x0, &full[st]);
            tma_load_2d(at + scales_at, &maps.w_scales, s * kTiles * 64, n0 / 128, &full[st]);
            tma_load_2d(at + scales_at + kWScales, &maps.x_scales, s * kTiles * 64, p.t0 / 128, &full[st]);
          }
        }
        __syncwarp();
        if (++st == a.stages) st = 0, ph ^= 1;
      }
    }
    if (!ok && lane == 0) s_bad = 1;
  } else if (warp == 1 && (CG == 1 || rank == 0)) {
    int st = 0, it = 0;
    uint32_t ph = 0;
    bool ok = true;
    const int per = (1 + a.x_tiles) * 4;  // TMEM columns of the scales of one tile of K
    for (int tile = first; tile < a.tiles && ok; tile += stride, ++it) {
      const Place p = place_of(a, tile);
      const uint32_t idesc = idesc_fp4<CG>(FMT == FT_FP4_MXFP4, columns_of<CG>(p.tokens));
      const int buf = a.buffers == 2 ? it & 1 : 0;
      const uint32_t acc = tmem + buf * (kScaleColumn / 2);
      if (it >= a.buffers) {
        if (!mbar_wait_warp<true>(&acc_empty[buf], (it / a.buffers - 1) & 1, a.status)) {
          ok = false;
          break;
        }
        tc_fence_after();
      }
      const uint32_t shift = (p.t0 & 127) >> 5;
      for (int s = s0; s < s1; ++s) {
        if (!mbar_wait_warp<true>(&full[st], ph, a.status)) {
          ok = false;
          break;
        }
        tc_fence_after();
        if (elect_one()) {
          const uint8_t* const at = smem + st * a.stage_bytes;
          const uint32_t cols = tmem + kScaleColumn + st * kTiles * per;  // [tile of K][weights, tokens 0.., tokens 128..][4]
          const uint64_t sc = scales_desc(at + scales_at);
#pragma unroll
          for (int i = 0; i < kTiles; ++i) {
            scales_to_tmem<CG>(cols + i * per, sc + i * 32);
            scales_to_tmem<CG>(cols + i * per + 4, sc + (kTiles + i) * 32);
            if (a.x_tiles == 2) scales_to_tmem<CG>(cols + i * per + 8, sc + (2 * kTiles + i) * 32);
          }
          const uint64_t wdesc = sw128_desc(at), xdesc = sw128_desc(at + x_at);
          const int n = min(4, (a.K - s * kStep + 63) / 64);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            if (j >= n) break;
            const uint32_t c = cols + (FMT == FT_FP4_MXFP4 ? j >> 1 : j) * per;
            mma_fp4<CG, FMT == FT_FP4_MXFP4>(acc, wdesc + 2 * j, xdesc + 2 * j,
                                             FMT == FT_FP4_MXFP4 ? idesc_scales(idesc, (j & 1) * 2) : idesc, c, c + 4 + shift,
                                             s > s0 || j > 0);
          }
          mma_commit<CG>(&empty[st]);
          if (s + 1 == s1) mma_commit<CG>(&acc_full[buf]);
        }
        __syncwarp();
        if (++st == a.stages) st = 0, ph ^= 1;
      }
    }
    if (!ok && lane == 0) s_bad = 1;
  } else if (warp >= 2) {
    const int e = warp - 2, q = warp & 3, h = e >> 2;  // the lanes that the warp may read; which chunks of 32 columns it takes
    const uint32_t empty_bar = CG == 2 ? map_cluster(smem_u32(&acc_empty[0]), 0) : smem_u32(&acc_empty[0]);
    const Fragment f = fragment_of(lane);
    uint8_t* const boxes = smem + a.stages * a.stage_bytes + (q * 2 + h) * (a.boxes * kBoxBytes);
    const uint32_t box0 = smem_u32(boxes);
    bool ok = true;
    int it = 0;
    // Seldom, a wait of an earlier call gave up, and nothing is written, or the warp's rows have far scales.  Those
    // are asked for a tile ahead, so that nothing waits for the answer.
    float own;  // the scale of row `lane` of the warp's
    const auto ask = [&](const Place& p) {
      const int n = p.w * kRows + (CG == 2 ? rank * kM : 0) + q * 32 + lane;
      // (slices: where they are joined)
      own = FMT == FT_FP4_NVFP4 && a.split == 1 && a.sw != nullptr && n < a.N ? a.sw[n * a.sw_stride] : 1.f;
    };
    const auto any_far = [&] { return __any_sync(0xffffffffu, far_scale(own)) != 0; };
    const int32_t found = status_now(a.status);
    ask(place_of(a, first));
    const bool gone = __any_sync(0xffffffffu, found == FT_ERR_TIMEOUT) != 0;
    bool seldom = any_far() || gone;
    for (int tile = first; tile < a.tiles && ok; tile += stride, ++it) {
      const Place p = place_of(a, tile);
      const int n0 = p.w * kRows + (CG == 2 ? rank * kM : 0) + q * 32;  // the warp's rows
      const int buf = a.buffers == 2 ? it & 1 : 0;
      const int mine = min(kChunks, (p.tokens - h * 32 + 63) / 64);  // chunks
      const uint32_t from = tmem + buf * (kScaleColumn / 2) + (static_cast<uint32_t>(q * 32) << 16) + h * 32;
      const auto release = [&] {  // the accumulator
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          if (CG == 2) mbar_arrive_cluster(empty_bar + buf * 8);
          else mbar_arrive(&acc_empty[buf]);
        }
      };
      if constexpr (BOXES) {
        if (lane == 0) {
          bulk_wait_read<0>();  // the boxes are free
          if (a.add != nullptr && mine > 0 && n0 < a.N) {
            mbar_arrive_expect_tx(&add_full[e], mine * kBoxBytes);
            for (int c = 0; c < mine; ++c)
              tma_load_2d(boxes + c * kBoxBytes, &maps.add, n0, p.t0 + (2 * c + h) * 32, &add_full[e]);
          }
        }
        __syncwarp();
      }
      ask(place_of(a, min(tile + stride, a.tiles - 1)));
      float sw[4], sx[kChunks];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int n = n0 + f.row + 8 * i;
        sw[i] = a.sw != nullptr && n < a.N ? a.sw[n * a.sw_stride] : 1.f;
      }
#pragma unroll
      for (int c = 0; c < kChunks; ++c) {
        const int t = (2 * c + h) * 32 + lane;
        sx[c] = a.sx != nullptr && t < p.tokens ? a.sx[(p.t0 + t) * a.sx_stride] : 1.f;
      }
      int kept = mine;  // chunks that are written
      const auto handle = [&] {
        if (gone) {
          kept = 0;
          if (lane == 0) s_skip = 1;
          return;
        }
        scale_in_tmem(from, mine, sw, a.sx == nullptr ? nullptr : a.sx + (p.t0 + h * 32) * a.sx_stride, a.sx_stride,
                      p.tokens - h * 32, f);
#pragma unroll
        for (int i = 0; i < 4; ++i) sw[i] = 1.f;
#pragma unroll
        for (int c = 0; c < kChunks; ++c) sx[c] = 1.f;
      };
      if constexpr (BOXES) {
        ok = mbar_wait_warp<true>(&acc_full[buf], (it / a.buffers) & 1, a.status);
        if (!ok) break;
        tc_fence_after();
        if (__builtin_expect(seldom, 0)) handle();
        uint32_t v[kChunks][32];
#pragma unroll
        for (int c = 0; c < kChunks; ++c)
          if (c < mine) tmem_ld32x32(from + c * 64, v[c]);
        tmem_wait();
        release();
        if (a.add != nullptr && mine > 0 && n0 < a.N) {
          ok = mbar_wait_warp<true>(&add_full[e], add_phase, a.status);
          if (!ok) break;
          add_phase ^= 1;
        }
#pragma unroll
        for (int c = 0; c < kChunks; ++c) {
          if (c >= kept) break;
          const int b = c & (a.boxes - 1);
          if (c >= a.boxes) {  // (no add: it has a box for each chunk)
            if (lane == 0) bulk_wait_read<1>();
            __syncwarp();
          }
          chunk_to_box<DT>(v[c], sw, sx[c], f, box0 + b * kBoxBytes, a.add != nullptr);
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0 && n0 < a.N) {
            tma_store_2d(&maps.out, n0, p.t0 + (2 * c + h) * 32, boxes + b * kBoxBytes);
            bulk_commit();
          }
        }
      } else {
        // A chunk at a time, the next one's add on its way; the first one's while the products run.
        Added<DT> add[2];
        const int t0 = p.t0 + h * 32;
        if (a.add != nullptr && mine > 0 && a.split == 1) load_added(a, t0, n0, f, add[0]);
        ok = mbar_wait_warp<true>(&acc_full[buf], (it / a.buffers) & 1, a.status);
        if (!ok) break;
        tc_fence_after();
        if (__builtin_expect(seldom, 0)) handle();
#pragma unroll
        for (int c = 0; c < kChunks; ++c) {
          if (c >= kept) break;
          uint32_t v[32];
          tmem_ld32x32(from + c * 64, v);
          if (a.add != nullptr && c + 1 < mine && a.split == 1) load_added(a, t0 + (c + 1) * 64, n0, f, add[(c + 1) & 1]);
          tmem_wait();
          if (c + 1 == kept) release();
          if (CG == 1 && a.split > 1) {
            float* const part = reinterpret_cast<float*>(smem);  // [token][kPartPitch]
#pragma unroll
            for (int i = 0; i < 32; ++i)
              part[((2 * c + h) * 32 + f.token(i)) * kPartPitch + q * 32 + f.row_of(i)] = __uint_as_float(v[i]);
          } else if (n0 + 32 <= a.N && t0 + c * 64 + 32 <= a.T) {
            chunk_to_rows<DT, true>(a, v, sw, sx[c], f, t0 + c * 64, n0, add[c & 1], box0);
          } else {
            chunk_to_rows<DT, false>(a, v, sw, sx[c], f, t0 + c * 64, n0, add[c & 1], box0);
          }
        }
        if (kept <= 0) release();
      }
      seldom = any_far() || gone;
    }
    if (lane == 0) {
      bulk_wait();
      if (!ok) s_bad = 1;
    }
  }
  if (CG == 1 && a.split > 1) {
    // the slices' partial sums: CTA `slice` joins its share of the elements
    const Place p = place_of(a, first);
    const int n = p.w * kM + lane * 4;
    __syncwarp();
    cluster_sync();
    float w_scale[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) w_scale[i] = a.sw != nullptr && n + i < a.N ? a.sw[(n + i) * a.sw_stride] : 1.f;
    uint32_t part[8];
#pragma unroll
    for (int r = 0; r < 8; ++r) part[r] = map_cluster(smem_u32(smem) + lane * 16, min(r, a.split - 1));
    const int tokens = s_skip != 0 ? 0 : p.tokens;
    // a token a warp: its 128 rows, four a lane
#pragma unroll 2
    for (int t = slice + a.split * warp; t < tokens; t += a.split * (kThreads / 32)) {
      const float sx = a.sx != nullptr ? a.sx[(p.t0 + t) * a.sx_stride] : 1.f;
      float4 x[8];
#pragma unroll
      for (int r = 0; r < 8; ++r) x[r] = r < a.split ? ld_cluster_f32x4(part[r] + t * (kPartPitch * 4)) : make_float4(0.f, 0.f, 0.f, 0.f);
      float y[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int r = 0; r < 8; ++r) y[0] += x[r].x, y[1] += x[r].y, y[2] += x[r].z, y[3] += x[r].w;
      float more[4];
      const int64_t to = (p.t0 + t) * a.out_stride + n, from = (p.t0 + t) * a.add_stride;
#pragma unroll
      for (int i = 0; i < 4; ++i) more[i] = a.add != nullptr ? load_out<DT>(a.add, from + min(n + i, a.N - 1)) : 0.f;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        asm volatile("" : "+f"(w_scale[i]));  // not to be split, and waited for, in front of the partial sums' loads
        const RowScale w = split_scale(w_scale[i]);
        y[i] = y[i] * w.near * sx * w.by;
        if (a.add != nullptr) y[i] += more[i];
        if (n + i < a.N) store_out<DT>(a.out, to + i, y[i]);
      }
    }
  }
  // A wait that gave up ends its role's loop with copies or products possibly
  // still in flight: let them land (a bounded 200 us) before TMEM is freed and
  // the CTA exits.
  tc_fence_before();
  __syncthreads();
  if (s_bad != 0) {
    const uint64_t t0 = global_timer_ns();
    while (global_timer_ns() - t0 < 200000ull) {
    }
  }
  __syncwarp();
  if (CG == 2 || a.split > 1) cluster_sync();  // nobody leaves while its memory or barriers are in use
  if (warp == 1) {
    tc_fence_after();
    tmem_free<CG>(tmem, 512);
  }
}

template <int FMT, int DT, int CG, bool BOXES>
ft_status launch(const Maps& maps, const MmArgs& a, cudaStream_t s) {
  const auto kernel = matmul_kernel<FMT, DT, CG, BOXES>;
  ft_status st = ensure_dyn_smem(reinterpret_cast<const void*>(kernel), kSmem, "fp4_matmul");
  if (st != FT_OK) return st;
  const int cluster = CG * a.split;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(std::min(a.tiles, device_sm_count() / cluster) * cluster);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kSmem;
  cfg.stream = s;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = cluster;
  at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 2;
  cudaLaunchKernelEx(&cfg, kernel, maps, a);
  return launch_check("fp4_matmul");
}

template <int FMT, int CG>
ft_status launch_typed(const Maps& maps, const MmArgs& a, int32_t dtype, bool by_boxes, cudaStream_t s) {
  switch (dtype) {
    case FT_DT_BF16:
      return by_boxes ? launch<FMT, FT_DT_BF16, CG, true>(maps, a, s) : launch<FMT, FT_DT_BF16, CG, false>(maps, a, s);
    case FT_DT_F16:
      return by_boxes ? launch<FMT, FT_DT_F16, CG, true>(maps, a, s) : launch<FMT, FT_DT_F16, CG, false>(maps, a, s);
    default: return launch<FMT, FT_DT_F32, CG, false>(maps, a, s);
  }
}

template <int FMT>
ft_status multiply(const Maps& maps, const MmArgs& a, int cg, int32_t dtype, bool by_boxes, cudaStream_t s) {
  return cg == 2 ? launch_typed<FMT, 2>(maps, a, dtype, by_boxes, s) : launch_typed<FMT, 1>(maps, a, dtype, by_boxes, s);
}

}  // namespace
}  // namespace ft
