// attn_e4m3.cu -- the decode attention kernel for 8-bit (E4M3) caches.
#include "ft_attend.cuh"

namespace ft {
ft_status attend_e4m3(AttnArgs& a, const AttnShape& sh, cudaStream_t s) {
  return launch_shape<FT_KV_E4M3>(a, sh, s);
}
}  // namespace ft
