// attn.cu -- ft_attn_decode: its checks, and the join of the partial sums that
// the attention kernels (ft_attend.cuh, one translation unit a cache format)
// leave where a unit of work crossed two workers' shares.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <math.h>

#include "ft_attn_args.cuh"

namespace ft {
namespace {

// Numbers of the line that the rows before `row` take, and all rows, by the
// whole block.
struct LineSums {
  int before, total;
};

template <int kThreads>
__device__ __forceinline__ LineSums line_sums(const AttnArgs& a, int row) {
  __shared__ int2 part_s[kThreads / 32];
  int before = 0, total = 0;
#pragma unroll 1
  for (int t = threadIdx.x; t < a.T; t += kThreads) {
    const int n = numbers_of(a, t);
    total += n;
    before += t < row ? n : 0;
  }
  before = __reduce_add_sync(0xffffffffu, before);
  total = __reduce_add_sync(0xffffffffu, total);
  if ((threadIdx.x & 31) == 0) part_s[threadIdx.x >> 5] = make_int2(before, total);
  __syncthreads();
  LineSums r = {0, 0};
#pragma unroll
  for (int w = 0; w < kThreads / 32; ++w) {
    r.before += part_s[w].x;
    r.total += part_s[w].y;
  }
  return r;
}

// Adds the partial sums of the unit that crosses the end of worker blockIdx.x's
// share and has its first tile in that share, in the workers' order.  A CTA
// takes kHeads heads of the block: one head with 16 warps (each every 16th
// partial) where few units have many partials each (one row of 130999 E4M3, one
// term a weight: 31.6 us in all, with 8 warps 33.1), eight heads with a warp each
// otherwise.
// Where there are fewer units than workers, CTA
// (x, y) takes unit x instead: most shares' ends are inside units that began
// before.
template <int kHeads>
constexpr int kJoinThreads = kHeads == 1 ? 512 : 256;

template <int DP, int kHeads>
__global__ void __launch_bounds__(kJoinThreads<kHeads>) join_kernel(const __grid_constant__ AttnArgs a) {
  constexpr int N = DP / 64;           // channel pairs of a lane: 2 * lane + 64 i
  constexpr int kThreads = kJoinThreads<kHeads>, kSpread = kThreads / 32 / kHeads;  // warps of a head
  constexpr int kBatch = kHeads == 1 ? (DP <= 128 ? 10 : 6) : 2;  // partials in flight
  __shared__ float2 acc_s[kSpread > 1 ? kSpread : 1][DP / 2];
  __shared__ float2 ml_s[kThreads / 32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int h = blockIdx.y * kHeads + warp / kSpread;
  // Which unit, and its workers, are worked out while they are at it: this grid
  // starts when attend_kernel's CTAs are past their own wait, so the lengths
  // are there.
  int t, unit, c0, c1;
  if (a.T * a.units <= a.workers) {
    t = blockIdx.x / a.units;
    unit = blockIdx.x - t * a.units;
    const LineSums line = line_sums<kThreads>(a, t);
    const int tiles = span_of(a, t).tiles, share = split_share(line.total, a.workers);
    const int from = line.before + unit * (tiles + a.lead) + a.lead;  // of its first tile
    c0 = from / share;
    c1 = tiles > 0 ? (from + tiles - 1) / share : c0;
  } else {
    const Begin end = begin_of<kThreads>(a, blockIdx.x + 1);
    t = end.t;
    c0 = c1 = blockIdx.x;
    unit = 0;
    if ((c0 + 1) * end.share < end.total) {
      const int tiles = span_of(a, t).tiles, n = tiles + a.lead;
      unit = end.at / n;
      const int held = end.at - unit * n - a.lead;  // its tiles before the share's end
      if (held > 0 && held <= end.share) c1 = c0 + (tiles - held + end.share - 1) / end.share;
    }
  }
  const int kv_head = unit / a.blocks;
  const int hg = (unit - kv_head * a.blocks) * a.block_heads + h;  // in the key head's group
  const bool live = h < a.block_heads && hg < a.G;
  // every CTA waits, whether it has something to add or not: work after this
  // grid must also come after attend_kernel
  pdl_wait();
  if (c0 == c1) return;
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
  const bool rows16 = a.kv.row_bytes == 2 * a.kv.D;
#pragma unroll
  for (int i = 0; i < N; ++i)
    if (2 * lane + 64 * i < a.kv.D) {
      const int64_t to = static_cast<int64_t>(t) * a.out_tok + static_cast<int64_t>(hq) * a.out_head + 2 * lane + 64 * i;
      float x = acc[i].x * inv, y = acc[i].y * inv;
      if (rows16) x = finite_or_nan(x), y = finite_or_nan(y);
      if (a.out_f32)
        *reinterpret_cast<float2*>(static_cast<float*>(a.out) + to) = make_float2(x, y);
      else
        *reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(a.out) + to) = pack_out(a, x, y);
    }
  if (lane == 0) store_lse(a, t, hq, m, l);
}

// ------------------------------------------------------------------ host side ---
int padded(int D) { return (D + 63) / 64 * 64; }
// 8-head column tiles of a warp: two where the group needs them and the
// accumulators (2 * DP * tiles / 32 registers a lane and head pair) leave room.
int head_tiles(int DP, int G) { return DP <= 128 && G > 8 ? 2 : 1; }

AttnShape shape_of(int D, int G) {
  AttnShape s;
  s.DP = padded(D);
  s.NT = head_tiles(s.DP, G);
  const int H = 8 * s.NT;
  s.columns = G > 2 * H ? 4 : G > H ? 2 : 1;
  s.block_heads = H * s.columns;
  s.blocks = (G + s.block_heads - 1) / s.block_heads;
  return s;
}

size_t part_o_bytes(const AttnShape& s) { return static_cast<size_t>(kMaxWorkers) * 2 * s.block_heads * s.DP * sizeof(float); }
size_t part_ml_bytes(const AttnShape& s) { return static_cast<size_t>(kMaxWorkers) * 2 * s.block_heads * sizeof(float2); }

template <int DP>
ft_status launch_join(const AttnArgs& a, cudaStream_t s) {
  const bool long_rows = a.workers > 8ll * a.T * a.units;  // more than eight partials a unit on average
  const int units = a.T * a.units;
  const dim3 grid(units < a.workers ? units : a.workers, long_rows ? a.block_heads : a.block_heads / 8);
  return launch_pdl(long_rows ? join_kernel<DP, 1> : join_kernel<DP, 8>, grid, long_rows ? kJoinThreads<1> : kJoinThreads<8>, 0, s, a, "attn_decode join");
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
  const AttnShape s = shape_of(D, Hq / Hkv);
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
  const AttnShape sh = shape_of(cache_host->D, Hq / Hkv);
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
  a.block_heads = sh.block_heads;
  // token positions stay well inside 31 bits (a tile past the last is computed)
  const int64_t most = static_cast<int64_t>(table_host->max_pages) * cache_host->page_size;
  a.most = static_cast<int32_t>(most < (1ll << 31) - 4096 ? most : (1ll << 31) - 4096);
  a.q_f16 = dtype == FT_DT_F16;
  a.out_f32 = out_dtype == FT_DT_F32;
  a.status = dev_status;
  cudaStream_t s = as_stream(stream);
  switch (fmt) {
    case FT_KV_BF16: st = attend_bf16(a, sh, s); break;
    case FT_KV_F16: st = attend_f16(a, sh, s); break;
    case FT_KV_E4M3: st = attend_e4m3(a, sh, s); break;
    default: st = attend_nvfp4(a, sh, s); break;
  }
  if (st != FT_OK) return st;
  switch (sh.DP) {
    case 64: return launch_join<64>(a, s);
    case 128: return launch_join<128>(a, s);
    case 192: return launch_join<192>(a, s);
    default: return launch_join<256>(a, s);
  }
}

}  // extern "C"
