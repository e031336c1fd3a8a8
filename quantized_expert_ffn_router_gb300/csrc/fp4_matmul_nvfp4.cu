// fp4_matmul_nvfp4.cu -- the products' kernels of the format FT_FP4_NVFP4.
#include "ft_fp4_matmul.cuh"

namespace ft {

ft_status multiply_nvfp4(const Maps& maps, const MmArgs& a, int cg, int32_t dtype, bool by_boxes, cudaStream_t s) {
  return multiply<FT_FP4_NVFP4>(maps, a, cg, dtype, by_boxes, s);
}

}  // namespace ft
