// ft_tensor.cuh -- the block-scaled 4-bit tensor core instructions, TMEM,
// tensor maps and clusters, as inline PTX for sm_103a.
#pragma once

#include <cuda.h>

#include "ft_async.cuh"

namespace ft {
namespace {

// ------------------------------------------------------------------ copies ---
__device__ __forceinline__ void prefetch_map(const CUtensorMap* map) {
  asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(map)) : "memory");
}

__device__ __forceinline__ void tma_load_2d(void* dst, const CUtensorMap* map, int c0, int c1, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3}], [%4];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(smem_u32(bar))
      : "memory");
}

// -------------------------------------------------------------------- TMEM ---
__device__ __forceinline__ void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }

// By one whole warp.
__device__ __forceinline__ void tmem_alloc(uint32_t* where, uint32_t columns) {
  asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(where)), "r"(columns)
               : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_free(uint32_t tmem, uint32_t columns) {
  asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(columns) : "memory");
}

#define FT_R8(b) "=r"(r[b]), "=r"(r[b + 1]), "=r"(r[b + 2]), "=r"(r[b + 3]), "=r"(r[b + 4]), "=r"(r[b + 5]), "=r"(r[b + 6]), "=r"(r[b + 7])
// 32 columns of the warp's 32 lanes.
__device__ __forceinline__ void tmem_ld32(uint32_t from, float (&v)[32]) {
  uint32_t r[32];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];\n"
      "tcgen05.wait::ld.sync.aligned;"
      : FT_R8(0), FT_R8(8), FT_R8(16), FT_R8(24)
      : "r"(from)
      : "memory");
#pragma unroll
  for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]);
}
#undef FT_R8

// ---------------------------------------------------------------- products ---
// K-major operand in the 128-byte swizzle: rows of 128 bytes, groups of 8 rows
// 1024 bytes apart, the tile 1024-byte aligned.
__device__ __forceinline__ uint64_t sw128_desc(const void* tile) {
  return ((smem_u32(tile) >> 4) & 0x3FFFull) | (1ull << 16) | (uint64_t{1024 >> 4} << 32) | (1ull << 46) | (2ull << 61);
}

// A scale tile: 32 rows of 16 bytes without swizzle, groups of 8 rows 128 bytes
// apart, copied to 32 lanes x 4 columns of each quarter of TMEM.
__device__ __forceinline__ void scales_to_tmem(uint32_t to, const void* tile) {
  const uint64_t d = ((smem_u32(tile) >> 4) & 0x3FFFull) | (uint64_t{128 >> 4} << 32) | (1ull << 46);
  asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(to), "l"(d) : "memory");
}

// E2M1 by E2M1, both K-major, M = 128, N = n: scales E4M3, or powers of two.
__device__ __forceinline__ uint32_t idesc_fp4(bool pow2, int n) {
  return (1u << 7) | (1u << 10) | (static_cast<uint32_t>(n >> 3) << 17) | (pow2 ? 1u << 23 : 0u) | (1u << 27);
}
// ... with the scales of a row from byte `id` of its word (powers of two: two of the four).
__device__ __forceinline__ uint32_t idesc_scales(uint32_t idesc, uint32_t id) { return idesc | (id << 4) | (id << 29); }

// 64 values of K.
template <bool POW2>
__device__ __forceinline__ void mma_fp4(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t sa, uint32_t sb,
                                        bool accumulate) {
  if (POW2)
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.b32 p, %6, 0;\n"
        " tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [%5], p;\n}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(sa), "r"(sb), "r"(static_cast<uint32_t>(accumulate))
        : "memory");
  else
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.b32 p, %6, 0;\n"
        " tcgen05.mma.cta_group::1.kind::mxf4nvf4.block_scale.scale_vec::4X [%0], %1, %2, %3, [%4], [%5], p;\n}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(sa), "r"(sb), "r"(static_cast<uint32_t>(accumulate))
        : "memory");
}

__device__ __forceinline__ void mma_commit(uint64_t* bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_u32(bar))
               : "memory");
}

// ---------------------------------------------------------------- clusters ---
// Every thread of every CTA of the cluster; stores before it are seen after it.
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// The float at a shared memory address of CTA `rank`.
__device__ __forceinline__ float ld_cluster_f32(uint32_t address, int rank) {
  uint32_t at;
  float v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(address), "r"(rank));
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(at) : "memory");
  return v;
}

// ----------------------------------------------------------- after a timeout ---
// A wait that gave up ends its role's loop with copies or products possibly
// still in flight: let them land (a bounded 200 us) before TMEM is freed and the
// CTA exits.  By the whole block.
__device__ __forceinline__ void drain_after_timeout(const int32_t* status) {
  __shared__ int s_drain;
  tc_fence_before();
  __syncthreads();
  if (threadIdx.x == 0)
    s_drain = status != nullptr && *reinterpret_cast<const volatile int32_t*>(status) == FT_ERR_TIMEOUT;
  __syncthreads();
  if (s_drain) {
    const uint64_t t0 = global_timer_ns();
    while (global_timer_ns() - t0 < 200000ull) {
    }
    __syncthreads();
  }
}

// ------------------------------------------------------------ tensor maps ---
using EncodeFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                              const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                              CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeFn encode_fn() {
  static const EncodeFn fn = [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      p = nullptr;
    return reinterpret_cast<EncodeFn>(p);
  }();
  return fn;
}

}  // namespace
}  // namespace ft
