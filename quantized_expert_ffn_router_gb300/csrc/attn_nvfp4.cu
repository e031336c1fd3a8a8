// attn_nvfp4.cu -- the decode attention kernel for 4-bit (NVFP4) caches.
#include "ft_attend.cuh"

namespace ft {
ft_status attend_nvfp4(AttnArgs& a, const AttnShape& sh, cudaStream_t s) {
  return launch_shape<FT_KV_NVFP4>(a, sh, s);
}
}  // namespace ft
