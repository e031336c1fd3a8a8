// fp4_matmul.cu -- the product of two microscaled 4-bit matrices, X [T, K] and
// W [N, K], on the block-scaled tensor cores.
//
// A tile is 128 rows of W (the M side, TMEM's lanes) by up to 256 tokens (the N
// side, its columns): one token's product then costs no more than the weights'
// bytes, and outputs are stored with 32 neighbouring n a warp, whatever the
// alignment of out.  A step is 256 values of K: 128 bytes of codes a row, by TMA
// in the 128-byte swizzle, and the scale tiles (512 bytes for 128 rows x 4
// scales) as they lie in memory, copied from shared memory to TMEM beside the
// accumulator in the same thread's order as the products that read them.
//
// Few tiles: K is cut into slices over the CTAs of a cluster, whose partial sums
// meet through distributed shared memory, added in the slices' order.
#include <cuda.h>

#include <algorithm>

#include "ft_fp4.cuh"
#include "ft_narrow.cuh"
#include "ft_tensor.cuh"

namespace ft {
namespace {

constexpr int kM = 128;          // weight rows of a tile
constexpr int kStep = 256;       // values of K in a step: four products of 64
constexpr int kThreads = 192;    // TMA, MMA, four warps of the epilogue
constexpr int kMaxStages = 8;
constexpr int kMaxWidth = 256;
constexpr int kSmem = 225 * 1024;

template <int FMT>
constexpr int step_tiles() { return FMT == FT_FP4_NVFP4 ? 4 : 2; }  // scale tiles of a step

struct MmArgs {
  void* out;
  const void* add;
  int64_t out_stride, add_stride;
  const float* sx;
  const float* sw;
  int64_t sx_stride, sw_stride;
  const uint8_t* x_scales;
  const uint8_t* w_scales;
  int32_t T, N, K;
  int32_t steps;    // of K
  int32_t ktiles;   // scale tiles of a row of tiles
  int32_t w_tiles;  // of 128 rows
  int32_t width;    // tokens of a tile
  int32_t split;    // CTAs of a cluster, slices of K
  int32_t stages, stage_bytes;
  int32_t dtype;
  int32_t* status;
};

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

template <int FMT, int DT>
__global__ void __launch_bounds__(kThreads, 1) matmul_kernel(const __grid_constant__ CUtensorMap wmap,
                                                             const __grid_constant__ CUtensorMap xmap,
                                                             const __grid_constant__ MmArgs a) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* const smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  __shared__ __align__(8) uint64_t full[kMaxStages], empty[kMaxStages], acc_full;
  __shared__ uint32_t s_tmem;
  constexpr int kTiles = step_tiles<FMT>();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = a.split > 1 ? static_cast<int>(blockIdx.x) % a.split : 0;
  const int tile = blockIdx.x / a.split;
  const int wt = tile % a.w_tiles, n0 = wt * kM;
  const int t0 = tile / a.w_tiles * a.width;
  const int tokens = min(a.width, a.T - t0);
  const int s0 = static_cast<int>(static_cast<int64_t>(a.steps) * rank / a.split);
  const int s1 = static_cast<int>(static_cast<int64_t>(a.steps) * (rank + 1) / a.split);
  const int x_tile0 = t0 / 128, x_tiles = (t0 + tokens + 127) / 128 - x_tile0;  // scale tiles of the tokens
  constexpr int kWBytes = kM * 128;
  const int x_bytes = a.width * 128;
  const uint32_t kAcc = kMaxWidth;  // TMEM columns: accumulators, then each stage's scales
  constexpr int kScaleCols = kTiles * 4 * 3;

  if (threadIdx.x == 0) {
    prefetch_map(&wmap);
    prefetch_map(&xmap);
    for (int i = 0; i < a.stages; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 1);
    }
    mbar_init(&acc_full, 1);
    fence_barrier_init();
  }
  if (warp == 1) tmem_alloc(&s_tmem, 512);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = s_tmem;
  pdl_wait();
  const bool skip = prior_timeout(a.status);
  bool ok = !skip;

  if (ok && warp == 0) {
    if (lane == 0) {
      int st = 0;
      uint32_t ph = 1;
      for (int s = s0; s < s1; ++s) {
        if (!mbar_wait(&empty[st], ph, a.status)) break;
        uint8_t* const at = smem + st * a.stage_bytes;
        const int nk = min(kTiles, a.ktiles - s * kTiles);
        mbar_arrive_expect_tx(&full[st], kWBytes + x_bytes + 512 * nk * (1 + x_tiles));
        tma_load_2d(at, &wmap, s * 128, n0, &full[st]);
        tma_load_2d(at + kWBytes, &xmap, s * 128, t0, &full[st]);
        uint8_t* const sc = at + kWBytes + x_bytes;
        bulk_g2s(sc, a.w_scales + (static_cast<int64_t>(wt) * a.ktiles + s * kTiles) * 512, 512 * nk, &full[st]);
        for (int i = 0; i < x_tiles; ++i)
          bulk_g2s(sc + (1 + i) * kTiles * 512, a.x_scales + (static_cast<int64_t>(x_tile0 + i) * a.ktiles + s * kTiles) * 512,
                   512 * nk, &full[st]);
        if (++st == a.stages) st = 0, ph ^= 1;
      }
    }
  } else if (ok && warp == 1) {
    if (lane == 0) {
      const uint32_t idesc = idesc_fp4(FMT == FT_FP4_MXFP4, (tokens + 15) & ~15);
      int st = 0;
      uint32_t ph = 0;
      bool good = true;
      for (int s = s0; s < s1; ++s) {
        if (!mbar_wait(&full[st], ph, a.status)) {
          good = false;
          break;
        }
        tc_fence_after();
        uint8_t* const at = smem + st * a.stage_bytes;
        const int nk = min(kTiles, a.ktiles - s * kTiles);
        const uint8_t* const sc = at + kWBytes + x_bytes;
        const uint32_t cols = tmem + kAcc + st * kScaleCols;  // [tile of K][weights, tokens 0.., tokens 128..][4]
        for (int i = 0; i < nk; ++i)
          for (int j = 0; j <= x_tiles; ++j)
            scales_to_tmem(cols + i * 12 + j * 4, sc + (j * kTiles + i) * 512);
        const uint64_t wdesc = sw128_desc(at), xdesc = sw128_desc(at + kWBytes);
        const int n = min(4, (a.K - s * kStep + 63) / 64);
        for (int j = 0; j < n; ++j) {
          const uint32_t c = cols + (FMT == FT_FP4_MXFP4 ? j >> 1 : j) * 12;
          mma_fp4<FMT == FT_FP4_MXFP4>(tmem, wdesc + 2 * j, xdesc + 2 * j,
                                       FMT == FT_FP4_MXFP4 ? idesc_scales(idesc, (j & 1) * 2) : idesc, c,
                                       c + 4 + ((t0 & 127) >> 5), s > s0 || j > 0);
        }
        mma_commit(&empty[st]);
        if (++st == a.stages) st = 0, ph ^= 1;
      }
      if (good) mma_commit(&acc_full);
    }
  } else if (ok) {
    const int q = warp & 3;  // the lanes that the warp may read
    if (!mbar_wait_warp(&acc_full, 0, a.status)) ok = false;
    if (ok) {
      tc_fence_after();
      const int row = q * 32 + lane, n = n0 + row;
      const uint32_t from = tmem + (static_cast<uint32_t>(q * 32) << 16);
      const float sw = a.sw != nullptr && n < a.N ? a.sw[n * a.sw_stride] : 1.f;
      float* const part = reinterpret_cast<float*>(smem);  // [token][128]
      for (int c0 = 0; c0 < tokens; c0 += 32) {
        float v[32];
        tmem_ld32(from + c0, v);
        if (a.split > 1) {
#pragma unroll
          for (int i = 0; i < 32; ++i)
            if (c0 + i < tokens) part[(c0 + i) * kM + row] = v[i];
          continue;
        }
        const int t = t0 + c0 + lane;
        const float sx_l = a.sx != nullptr && t < a.T ? a.sx[t * a.sx_stride] : 1.f;
#pragma unroll
        for (int i = 0; i < 32; ++i) {
          const float sx = __shfl_sync(0xffffffffu, sx_l, i);
          if (c0 + i >= tokens || n >= a.N) continue;
          float y = v[i] * sw * sx;
          const int64_t t_at = t0 + c0 + i;
          if (a.add != nullptr) y += load_out<DT>(a.add, t_at * a.add_stride + n);
          store_out<DT>(a.out, t_at * a.out_stride + n, y);
        }
      }
    }
    tc_fence_before();
  }
  if (a.split > 1) {
    // the slices' partial sums: CTA `rank` joins its share of the elements
    __syncwarp();
    cluster_sync();
    const int total = tokens * kM, share = (total + a.split - 1) / a.split;
    const uint32_t mine = smem_u32(smem);
    for (int e = rank * share + threadIdx.x; e < min(total, (rank + 1) * share); e += kThreads) {
      float y = 0.f;
      for (int r = 0; r < a.split; ++r) y += ld_cluster_f32(mine + e * 4, r);
      const int n = n0 + e % kM;
      const int64_t t = t0 + e / kM;
      if (n >= a.N) continue;
      y *= a.sw != nullptr ? a.sw[n * a.sw_stride] : 1.f;
      y *= a.sx != nullptr ? a.sx[t * a.sx_stride] : 1.f;
      if (a.add != nullptr) y += load_out<DT>(a.add, t * a.add_stride + n);
      store_out<DT>(a.out, t * a.out_stride + n, y);
    }
    cluster_sync();
  }
  drain_after_timeout(a.status);
  if (warp == 1) {
    tc_fence_after();
    tmem_free(tmem, 512);
  }
}

// A matrix's codes, in boxes of 128 bytes by so many rows.
bool map_codes(CUtensorMap* map, const ft_fp4_matrix* m, int rows) {
  const cuuint64_t dims[2] = {static_cast<cuuint64_t>(m->K / 2), static_cast<cuuint64_t>(m->rows)};
  const cuuint64_t strides[1] = {static_cast<cuuint64_t>(m->pitch)};
  const cuuint32_t box[2] = {128, static_cast<cuuint32_t>(rows)};
  const cuuint32_t es[2] = {1, 1};
  return encode_fn()(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, m->codes, dims, strides, box, es,
                     CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                     CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int FMT, int DT>
ft_status launch(const CUtensorMap& wmap, const CUtensorMap& xmap, const MmArgs& a, int64_t tiles, cudaStream_t s) {
  const auto kernel = matmul_kernel<FMT, DT>;
  ft_status st = ensure_dyn_smem(reinterpret_cast<const void*>(kernel), kSmem, "fp4_matmul");
  if (st != FT_OK) return st;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(tiles * a.split));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kSmem;
  cfg.stream = s;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = a.split;
  at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 2;
  cudaLaunchKernelEx(&cfg, kernel, wmap, xmap, a);
  return launch_check("fp4_matmul");
}

template <int FMT>
ft_status launch_typed(const CUtensorMap& w, const CUtensorMap& x, const MmArgs& a, int64_t tiles, cudaStream_t s) {
  switch (a.dtype) {
    case FT_DT_BF16: return launch<FMT, FT_DT_BF16>(w, x, a, tiles, s);
    case FT_DT_F16: return launch<FMT, FT_DT_F16>(w, x, a, tiles, s);
    default: return launch<FMT, FT_DT_F32>(w, x, a, tiles, s);
  }
}

}  // namespace
}  // namespace ft

using namespace ft;

extern "C" {

ft_status ft_fp4_matmul(const ft_fp4_matrix* x_host, const ft_fp4_matrix* w_host, void* out, int64_t out_stride,
                        int32_t dtype, const void* add, int64_t add_stride, int32_t* dev_status, void* stream) {
  const char* what = "fp4_matmul";
  ft_status st;
  if ((st = check_fp4(what, "x", x_host)) != FT_OK) return st;
  if ((st = check_fp4(what, "w", w_host)) != FT_OK) return st;
  FT_REQUIRE(x_host->fmt == w_host->fmt, "%s: x and w are of different formats", what);
  FT_REQUIRE(x_host->K == w_host->K, "%s: K is %lld in x and %lld in w", what, static_cast<long long>(x_host->K),
             static_cast<long long>(w_host->K));
  if (x_host->order != FT_FP4_TILES || w_host->order != FT_FP4_TILES)
    return fail(FT_ERR_UNSUPPORTED, "%s: block scales must be in the order FT_FP4_TILES", what);
  FT_REQUIRE(dtype >= FT_DT_BF16 && dtype <= FT_DT_F32, "%s: dtype %d", what, dtype);
  if (x_host->rows == 0 || w_host->rows == 0) return FT_OK;
  const uintptr_t size = dtype == FT_DT_F32 ? 4 : 2;
  FT_REQUIRE(out != nullptr && reinterpret_cast<uintptr_t>(out) % size == 0, "%s: out is NULL or not aligned", what);
  FT_REQUIRE(reinterpret_cast<uintptr_t>(add) % size == 0, "%s: add is not aligned", what);
  FT_REQUIRE(out_stride >= 0 && add_stride >= 0, "%s: negative stride", what);
  FT_REQUIRE(add != out || add_stride == out_stride, "%s: in place needs the same strides", what);
  if (encode_fn() == nullptr) return fail(FT_ERR_CUDA, "%s: cuTensorMapEncodeTiled unavailable", what);
  MmArgs a = {};
  a.out = out;
  a.add = add;
  a.out_stride = out_stride;
  a.add_stride = add_stride;
  a.sx = x_host->scale;
  a.sw = w_host->scale;
  a.sx_stride = x_host->scale_stride;
  a.sw_stride = w_host->scale_stride;
  a.x_scales = x_host->scales;
  a.w_scales = w_host->scales;
  a.T = static_cast<int32_t>(x_host->rows);
  a.N = static_cast<int32_t>(w_host->rows);
  a.K = static_cast<int32_t>(x_host->K);
  a.steps = static_cast<int32_t>((x_host->K + kStep - 1) / kStep);
  a.ktiles = static_cast<int32_t>((x_host->K / fp4_block(x_host->fmt) + 3) / 4);
  a.w_tiles = (a.N - 1) / kM + 1;
  a.dtype = dtype;
  a.status = dev_status;
  const int sms = device_sm_count();
  const auto tiles_of = [&](int width) { return static_cast<int64_t>(a.w_tiles) * ((a.T - 1) / width + 1); };
  a.split = 1;
  if (a.T <= 64) {
    a.width = (a.T + 15) / 16 * 16;
  } else {
    // waves of the SMs times what a tile takes
    double best = 0;
    for (int w = 64; w <= kMaxWidth; w += 64) {
      const double cost = static_cast<double>((tiles_of(w) + sms - 1) / sms) * (w + 64);
      if (w == 64 || cost <= best) best = cost, a.width = w;
    }
  }
  const int64_t tiles = tiles_of(a.width);
  while (a.split < 8 && tiles * a.split * 2 <= sms && a.split * 2 <= a.steps) a.split *= 2;
  FT_REQUIRE(tiles * a.split < (1ll << 31), "%s: too many tiles", what);
  a.stage_bytes = kM * 128 + a.width * 128 + (x_host->fmt == FT_FP4_NVFP4 ? 2048 : 1024) * 3;
  a.stages = std::min((kSmem - 1024) / a.stage_bytes, std::min(kMaxStages, 256 / (x_host->fmt == FT_FP4_NVFP4 ? 48 : 24)));
  CUtensorMap wmap, xmap;
  if (!map_codes(&wmap, w_host, kM) || !map_codes(&xmap, x_host, a.width))
    return fail(FT_ERR_INVALID, "%s: a tensor map of the codes was rejected", what);
  cudaStream_t s = as_stream(stream);
  return x_host->fmt == FT_FP4_NVFP4 ? launch_typed<FT_FP4_NVFP4>(wmap, xmap, a, tiles, s)
                                     : launch_typed<FT_FP4_MXFP4>(wmap, xmap, a, tiles, s);
}

}  // extern "C"
