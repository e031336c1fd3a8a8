// ft_fp4.cuh -- microscaled 4-bit matrices: what the host checks of the public
// descriptors share.
#pragma once

#include "ft_async.cuh"
#include "ft_common.cuh"
#include "ft_fp4.h"

namespace ft {

constexpr int64_t kScaleTileRows = 128, kScaleTileBlocks = 4;  // of the order FT_FP4_TILES, 512 bytes

constexpr int fp4_block(int fmt) { return fmt == FT_FP4_NVFP4 ? 16 : 32; }

// Calls of at most so many rows let the next kernel be set up while they run
// (quantise and project 1 x 2560 x 2048 in a graph: 6.7 us, then 5.9; 8 x 4096 x
// 4096: 7.4, then 6.7).  Longer ones do not: what is set up on an SM that a product
// has left no L1 on keeps it so (quantise and project 2048 x 4096 x 4096: 27.3 us,
// then 28.8).  A long product of few rows has both: 64 x 131072 x 2048 and, behind it,
// itself 28.7 us, then 27.9 each, a product of 2048 x 4096 x 4096 together 49.4, then
// 47.5; quantising 64 rows 30.0, then 30.6, 4096 rows 40.8, then 43.7; another program's
// kernel that does not ask for it, no difference.
constexpr int64_t kFewRows = 64;

// Refuses descriptors that the kernels must not see; a matrix of no rows needs no memory.
ft_status check_fp4(const char* what, const char* name, const ft_fp4_matrix* m);

}  // namespace ft
