// ft_fp4.cuh -- microscaled 4-bit matrices: what the host checks of the public
// descriptors share.
#pragma once

#include "ft_async.cuh"
#include "ft_common.cuh"
#include "ft_fp4.h"

namespace ft {

constexpr int64_t kScaleTileRows = 128, kScaleTileBlocks = 4;  // of the order FT_FP4_TILES, 512 bytes

constexpr int fp4_block(int fmt) { return fmt == FT_FP4_NVFP4 ? 16 : 32; }

// Refuses descriptors that the kernels must not see; a matrix of no rows needs no memory.
ft_status check_fp4(const char* what, const char* name, const ft_fp4_matrix* m);

}  // namespace ft
