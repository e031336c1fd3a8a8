// attn_f16.cu -- the decode attention kernel for f16 caches.
#include "ft_attend.cuh"

namespace ft {
ft_status attend_f16(AttnArgs& a, const AttnShape& sh, cudaStream_t s) {
  return launch_shape<FT_KV_F16>(a, sh, s);
}
}  // namespace ft
