// ft_attn_args.cuh -- what attn.cu and the attention kernels share: the
// arguments, the shapes, and the launch of each format's kernel.
#pragma once

#include "ft_kv.cuh"

namespace ft {

constexpr int kMaxWorkers = 1024;  // CTAs of one call (sizes the workspace)

struct AttnArgs {
  KvView kv;
  const uint16_t* q;
  int64_t q_tok, q_head;
  void* out;
  int64_t out_tok, out_head;
  float* lse;
  const int32_t* lens;
  float* part_o;   // [worker][2][heads of a block][D padded]
  float2* part_ml;  // [worker][2][heads of a block] (maximum, sum)
  float scale_log2;
  int32_t window, T, Hq, G;
  int32_t units;         // head blocks of a row: Hkv * blocks
  int32_t blocks;        // head blocks of a key head
  int32_t warps_h_log2;  // warps of a CTA over head tiles; the others over tokens
  int32_t block_heads;   // heads of a block
  int32_t tile;          // tokens of a CTA's tile
  int32_t lead;          // numbers of a unit in the line before those of its tiles
  int32_t most;          // max_pages * page_size
  int32_t q_f16, out_f32;
  int32_t workers;
  int32_t* status;
};

__device__ __forceinline__ RowSpan span_of(const AttnArgs& a, int t) {
  return row_span(a.lens[t], a.window, a.most, a.tile);
}

// Numbers of the line that the rows before `rows` take, by one warp.
__device__ __forceinline__ int numbers_before(const AttnArgs& a, int rows, int lane) {
  int n = 0;
  for (int t = lane; t < rows; t += 32) n += row_numbers(span_of(a, t).tiles, a.lead, a.units);
  return __reduce_add_sync(0xffffffffu, n);
}

struct AttnShape {
  int DP, NT;        // channels padded to 64s; 8-head column tiles of a warp
  int warps_h_log2, block_heads, blocks;
};

// The kernel of each cache format; sets a.tile and a.workers.
ft_status attend_bf16(AttnArgs& a, const AttnShape& sh, cudaStream_t s);
ft_status attend_f16(AttnArgs& a, const AttnShape& sh, cudaStream_t s);
ft_status attend_e4m3(AttnArgs& a, const AttnShape& sh, cudaStream_t s);
ft_status attend_nvfp4(AttnArgs& a, const AttnShape& sh, cudaStream_t s);

}  // namespace ft
