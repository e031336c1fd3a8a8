// ft_fp4_args.cuh -- what fp4_matmul.cu and the products' kernels share: the
// tiles, the arguments, and the launch of each format's kernels.
#pragma once

#include <cuda.h>

#include "ft_fp4.cuh"
#include "ft_fp4_tiles.h"

namespace ft {

constexpr int kEpilogueWarps = 8;
constexpr int kThreads = 64 + 32 * kEpilogueWarps;  // TMA, MMA, epilogue
constexpr int kMaxStages = 8;
constexpr int kScaleColumn = 256;  // of TMEM: accumulators before it, each stage's scales from it
constexpr int kChunks = kMaxWidth / 32 / 2;  // of 32 columns that a warp of the epilogue takes, at most
constexpr int kBoxBytes = 32 * 64;  // 32 tokens x 32 rows of 16-bit outputs
constexpr int kPartPitch = kM + 4;  // floats of a token's partial sums: fragments are stored without bank conflicts
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
  int32_t T, N, K;
  int32_t steps;    // of K
  int32_t tiles;
  int32_t inner;    // tiles that follow one another share the outer matrix's rows: this many, ...
  int32_t x_inner;  // ... of tokens (the smaller matrix goes round inside)
  int32_t width;    // tokens of a tile
  int32_t x_tiles;  // scale tiles that a tile's tokens lie in, at most
  int32_t buffers;  // accumulators
  int32_t split;    // slices of K, one a CTA of a cluster (pairs of CTAs: 1)
  int32_t stages, stage_bytes;
  int32_t boxes;    // of 32 tokens that each warp of the epilogue has in shared memory, a power of two
  int32_t words;    // row by row: out and add hold whole words of two rows
  int32_t* status;
};

struct Maps {
  CUtensorMap w, x, w_scales, x_scales, out, add;
};

// The kernels of each format: pairs of CTAs or single ones, out by boxes or row by row.
ft_status multiply_nvfp4(const Maps& maps, const MmArgs& a, int cg, int32_t dtype, bool by_boxes, cudaStream_t s);
ft_status multiply_mxfp4(const Maps& maps, const MmArgs& a, int cg, int32_t dtype, bool by_boxes, cudaStream_t s);

}  // namespace ft
