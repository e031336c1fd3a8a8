// fp4_matmul.cu -- ft_fp4_matmul's entry point: checks and tensor maps.  The choice
// of tiles: ft_fp4_tiles.h; the kernels: ft_fp4_matmul.cuh.
#include <algorithm>

#include "ft_fp4_args.cuh"
#include "ft_tensor.cuh"

namespace ft {
namespace {

constexpr int64_t kMostRows = (1ll << 31) - 1024;

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

// Its scale tiles: a row of tiles in 8-byte words, in boxes of a step by so many rows of tiles.
bool map_scales(CUtensorMap* map, const ft_fp4_matrix* m, int64_t ktiles, int step, int rows) {
  const cuuint64_t dims[2] = {static_cast<cuuint64_t>(ktiles * 64),
                              static_cast<cuuint64_t>((m->rows + kScaleTileRows - 1) / kScaleTileRows)};
  const cuuint64_t strides[1] = {static_cast<cuuint64_t>(ktiles * 512)};
  const cuuint32_t box[2] = {static_cast<cuuint32_t>(step * 64), static_cast<cuuint32_t>(rows)};
  const cuuint32_t es[2] = {1, 1};
  return encode_fn()(map, CU_TENSOR_MAP_DATA_TYPE_INT64, 2, m->scales, dims, strides, box, es,
                     CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                     CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Rows of 16-bit outputs, in boxes of 32 by 32 tokens.
bool map_rows(CUtensorMap* map, const void* p, int64_t N, int64_t T, int64_t stride) {
  const cuuint64_t dims[2] = {static_cast<cuuint64_t>(N), static_cast<cuuint64_t>(T)};
  // one row may have any stride
  const cuuint64_t strides[1] = {static_cast<cuuint64_t>(T > 1 ? stride * 2 : (N + 7) / 8 * 16)};
  const cuuint32_t box[2] = {32, 32};
  const cuuint32_t es[2] = {1, 1};
  return encode_fn()(map, CU_TENSOR_MAP_DATA_TYPE_UINT16, 2, const_cast<void*>(p), dims, strides, box, es,
                     CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_64B, CU_TENSOR_MAP_L2_PROMOTION_NONE,
                     CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
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
  // rows are numbered in 32 bits, up to the end of the last tile
  if (x_host->rows > kMostRows || w_host->rows > kMostRows)
    return fail(FT_ERR_UNSUPPORTED, "%s: more than %lld rows", what, static_cast<long long>(kMostRows));
  FT_REQUIRE(dtype >= FT_DT_BF16 && dtype <= FT_DT_F32, "%s: dtype %d", what, dtype);
  if (x_host->rows == 0 || w_host->rows == 0) return FT_OK;
  const uintptr_t size = dtype == FT_DT_F32 ? 4 : 2;
  FT_REQUIRE(out != nullptr && reinterpret_cast<uintptr_t>(out) % size == 0, "%s: out is NULL or not aligned", what);
  FT_REQUIRE(reinterpret_cast<uintptr_t>(add) % size == 0, "%s: add is not aligned", what);
  FT_REQUIRE(out_stride >= 0 && add_stride >= 0, "%s: negative stride", what);
  FT_REQUIRE(x_host->rows == 1 || out_stride >= w_host->rows, "%s: rows of out overlap", what);
  FT_REQUIRE(add != out || add_stride == out_stride || x_host->rows == 1, "%s: in place needs the same strides", what);
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
  a.T = static_cast<int32_t>(x_host->rows);
  a.N = static_cast<int32_t>(w_host->rows);
  a.K = static_cast<int32_t>(x_host->K);
  a.steps = static_cast<int32_t>((x_host->K + kStep - 1) / kStep);
  a.status = dev_status;
  const auto whole = [](const void* p, int64_t stride) { return reinterpret_cast<uintptr_t>(p) % 16 == 0 && stride % 8 == 0; };
  // (a tensor map has no rows that overlap, such as one row added to all tokens)
  bool by_boxes = dtype != FT_DT_F32 && whole(out, out_stride) &&
                  (add == nullptr || (whole(add, add_stride) && (a.T == 1 || add_stride >= a.N)));
  const auto even = [](const void* p, int64_t stride) { return reinterpret_cast<uintptr_t>(p) % 4 == 0 && stride % 2 == 0; };
  a.words = dtype != FT_DT_F32 && a.N % 2 == 0 && even(out, out_stride) && (add == nullptr || even(add, add_stride));
  const bool nv = x_host->fmt == FT_FP4_NVFP4;
  const int sms = device_sm_count(), step = nv ? step_tiles<FT_FP4_NVFP4>() : step_tiles<FT_FP4_MXFP4>();
  const Tiles t = choose_tiles(a.T, a.N, a.steps, sms);
  const int cg = t.pair;
  a.width = t.width;
  a.split = t.slices;
  const int64_t tiles = tiles_of(a.T, a.N, a.width, cg);
  FT_REQUIRE(tiles < (1ll << 31), "%s: too many tiles", what);
  a.tiles = static_cast<int32_t>(tiles);
  by_boxes = by_boxes && a.split == 1;  // the slices' sums are joined and written otherwise
  a.x_inner = a.T <= a.N;
  a.inner = a.x_inner ? (a.T - 1) / a.width + 1 : (a.N - 1) / (kM * cg) + 1;
  a.x_tiles = a.width > 128 ? 2 : 1;
  a.buffers = a.width > 128 ? 1 : 2;
  a.stage_bytes = kM * 128 + a.width / cg * 128 + step * 512 * (1 + a.x_tiles);
  a.stage_bytes = (a.stage_bytes + 1023) & ~1023;
  // two boxes a warp (row by row: one); add is loaded ahead, into one for each chunk
  const int chunks = (a.width + 63) / 64;
  a.boxes = !by_boxes ? 1 : add == nullptr ? std::min(chunks, 2) : chunks > 2 ? 4 : chunks;
  const int boxes = dtype == FT_DT_F32 ? 0 : kEpilogueWarps * a.boxes * kBoxBytes;
  a.stages = std::min({(kSmem - 1024 - boxes) / a.stage_bytes, kMaxStages, (512 - kScaleColumn) / (step * 4 * (1 + a.x_tiles))});
  const int64_t ktiles = (x_host->K / fp4_block(x_host->fmt) + 3) / 4;
  Maps maps;
  if (!map_codes(&maps.w, w_host, kM) || !map_codes(&maps.x, x_host, a.width / cg) ||
      !map_scales(&maps.w_scales, w_host, ktiles, step, 1) || !map_scales(&maps.x_scales, x_host, ktiles, step, a.x_tiles))
    return fail(FT_ERR_INVALID, "%s: a tensor map of the codes or scales was rejected", what);
  if (by_boxes && (!map_rows(&maps.out, out, a.N, a.T, out_stride) ||
                   (add != nullptr && !map_rows(&maps.add, add, a.N, a.T, add_stride))))
    return fail(FT_ERR_INVALID, "%s: a tensor map of out or add was rejected", what);
  cudaStream_t s = as_stream(stream);
  return (nv ? multiply_nvfp4 : multiply_mxfp4)(maps, a, cg, dtype, by_boxes, s);
}

}  // extern "C"
