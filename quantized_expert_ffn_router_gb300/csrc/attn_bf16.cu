// attn_bf16.cu -- the decode attention kernel for bf16 caches.
#include "ft_attend.cuh"

namespace ft {
ft_status attend_bf16(AttnArgs& a, const AttnShape& sh, cudaStream_t s) {
  return launch_shape<FT_KV_BF16>(a, sh, s);
}
}  // namespace ft
