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

// The same by a CTA of a pair, counted on the barrier of either (a shared::cluster address).
__device__ __forceinline__ void tma_load_2d_pair(void* dst, const CUtensorMap* map, int c0, int c1, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3}], [%4];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(bar)
      : "memory");
}

// A box from shared memory, in the thread's bulk group.
__device__ __forceinline__ void tma_store_2d(const CUtensorMap* map, int c0, int c1, const void* src) {
  asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.tile.bulk_group [%0, {%1, %2}], [%3];" ::"l"(
                   reinterpret_cast<uint64_t>(map)),
               "r"(c0), "r"(c1), "r"(smem_u32(src))
               : "memory");
}
__device__ __forceinline__ void bulk_commit() { asm volatile("cp.async.bulk.commit_group;" ::: "memory"); }
// The thread's stores, but the last LEFT, have read shared memory (`bulk_wait`: all are done).
template <int LEFT>
__device__ __forceinline__ void bulk_wait_read() { asm volatile("cp.async.bulk.wait_group.read %0;" ::"n"(LEFT) : "memory"); }
__device__ __forceinline__ void bulk_wait() { asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); }
__device__ __forceinline__ void fence_proxy_async_smem() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

// Four 8 x 8 matrices of 16-bit values, transposed: lane 8 j + i has the address
// of row i of matrix j in memory; register j holds column `lane` / 4, rows
// 2 (lane % 4) and the next.
__device__ __forceinline__ void store_transposed(uint32_t at, const uint32_t (&r)[4]) {
  asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(r[0]), "r"(r[1]),
               "r"(r[2]), "r"(r[3])
               : "memory");
}
__device__ __forceinline__ void load_transposed(uint32_t at, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(at)
               : "memory");
}

// Not to be moved over stores of shared memory, but over those of global memory.
__device__ __forceinline__ uint32_t ld_shared_u32(uint32_t at) {
  uint32_t x;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(x) : "r"(at));
  return x;
}
__device__ __forceinline__ uint16_t ld_shared_u16(uint32_t at) {
  uint16_t x;
  asm volatile("ld.shared.u16 %0, [%1];" : "=h"(x) : "r"(at));
  return x;
}

__device__ __forceinline__ void st_shared_u32(uint32_t at, uint32_t x) {
  asm volatile("st.shared.u32 [%0], %1;" ::"r"(at), "r"(x) : "memory");
}
__device__ __forceinline__ void st_shared_u16(uint32_t at, uint16_t x) {
  asm volatile("st.shared.u16 [%0], %1;" ::"r"(at), "h"(x) : "memory");
}

// One lane of a warp that runs together.
__device__ __forceinline__ bool elect_one() {
  uint32_t is;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}" : "=r"(is));
  return is != 0;
}

// -------------------------------------------------------------------- TMEM ---
__device__ __forceinline__ void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }

// By one whole warp; CG 2: of each CTA of a pair.
template <int CG>
__device__ __forceinline__ void tmem_alloc(uint32_t* where, uint32_t columns) {
  if (CG == 2) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(where)), "r"(columns)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  } else {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(where)), "r"(columns)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
}
template <int CG>
__device__ __forceinline__ void tmem_free(uint32_t tmem, uint32_t columns) {
  if (CG == 2)
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(columns) : "memory");
  else
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(columns) : "memory");
}

#define FT_R8(b) "=r"(r[b]), "=r"(r[b + 1]), "=r"(r[b + 2]), "=r"(r[b + 3]), "=r"(r[b + 4]), "=r"(r[b + 5]), "=r"(r[b + 6]), "=r"(r[b + 7])
// 32 columns of 16 lanes, in flight until tmem_wait: of columns 8 k + 2 (lane % 4)
// and the next, r[4 k], r[4 k + 1] are TMEM lane `lane` / 4, r[4 k + 2], r[4 k + 3]
// the one 8 further.
__device__ __forceinline__ void tmem_ld16x32(uint32_t from, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x4.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : FT_R8(0), FT_R8(8)
      : "r"(from)
      : "memory");
}
#undef FT_R8
// 8 columns of 16 lanes, likewise.
__device__ __forceinline__ void tmem_ld16x8(uint32_t from, uint32_t (&r)[4]) {
  asm volatile("tcgen05.ld.sync.aligned.16x256b.x1.b32 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(from)
               : "memory");
}
// The same the other way, in flight until tmem_wait_stores.
__device__ __forceinline__ void tmem_st16x8(uint32_t to, const uint32_t (&r)[4]) {
  asm volatile("tcgen05.st.sync.aligned.16x256b.x1.b32 [%4], {%0, %1, %2, %3};" ::"r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(to)
               : "memory");
}
__device__ __forceinline__ void tmem_wait_stores() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tmem_wait() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }

// ---------------------------------------------------------------- products ---
// K-major operand in the 128-byte swizzle: rows of 128 bytes, groups of 8 rows
// 1024 bytes apart, the tile 1024-byte aligned.
__device__ __forceinline__ uint64_t sw128_desc(const void* tile) {
  return ((smem_u32(tile) >> 4) & 0x3FFFull) | (1ull << 16) | (uint64_t{1024 >> 4} << 32) | (1ull << 46) | (2ull << 61);
}

// A scale tile: 32 rows of 16 bytes without swizzle, groups of 8 rows 128 bytes
// apart, copied to 32 lanes x 4 columns of each quarter of TMEM (CG 2: by each
// CTA of the pair from its own shared memory to its own TMEM).
__device__ __forceinline__ uint64_t scales_desc(const void* tile) {
  return ((smem_u32(tile) >> 4) & 0x3FFFull) | (uint64_t{128 >> 4} << 32) | (1ull << 46);
}
template <int CG>
__device__ __forceinline__ void scales_to_tmem(uint32_t to, uint64_t desc) {
  if (CG == 2)
    asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;" ::"r"(to), "l"(desc) : "memory");
  else
    asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(to), "l"(desc) : "memory");
}

// E2M1 by E2M1, both K-major, M = 128 (CG 2: 256), N = n: scales E4M3, or powers of two.
template <int CG>
__device__ __forceinline__ uint32_t idesc_fp4(bool pow2, int n) {
  return (1u << 7) | (1u << 10) | (static_cast<uint32_t>(n >> 3) << 17) | (pow2 ? 1u << 23 : 0u) | (uint32_t{CG} << 27);
}
// ... with the scales of a row from byte `id` of its word (powers of two: two of the four).
__device__ __forceinline__ uint32_t idesc_scales(uint32_t idesc, uint32_t id) { return idesc | (id << 4) | (id << 29); }

#define FT_MMA(GROUP, KIND)                                                                                            \
  asm volatile("{\n .reg .pred p;\n setp.ne.b32 p, %6, 0;\n tcgen05.mma." GROUP "." KIND                               \
               " [%0], %1, %2, %3, [%4], [%5], p;\n}" ::"r"(d),                                                         \
               "l"(a), "l"(b), "r"(idesc), "r"(sa), "r"(sb), "r"(static_cast<uint32_t>(accumulate))                      \
               : "memory")
// 64 values of K.
template <int CG, bool POW2>
__device__ __forceinline__ void mma_fp4(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t sa, uint32_t sb,
                                        bool accumulate) {
  if (CG == 2) {
    if (POW2) FT_MMA("cta_group::2", "kind::mxf4.block_scale.scale_vec::2X");
    else FT_MMA("cta_group::2", "kind::mxf4nvf4.block_scale.scale_vec::4X");
  } else {
    if (POW2) FT_MMA("cta_group::1", "kind::mxf4.block_scale.scale_vec::2X");
    else FT_MMA("cta_group::1", "kind::mxf4nvf4.block_scale.scale_vec::4X");
  }
}
#undef FT_MMA

// The barrier (of both CTAs of a pair) is arrived at once the products issued so far are done.
template <int CG>
__device__ __forceinline__ void mma_commit(uint64_t* bar) {
  if (CG == 2)
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
            smem_u32(bar)),
        "h"(static_cast<uint16_t>(3))
        : "memory");
  else
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_u32(bar))
                 : "memory");
}

// ---------------------------------------------------------------- clusters ---
// Every thread of every CTA of the cluster; stores before it are seen after it.
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}

// A shared memory address in CTA `rank`.
__device__ __forceinline__ uint32_t map_cluster(uint32_t address, uint32_t rank) {
  uint32_t at;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(address), "r"(rank));
  return at;
}

__device__ __forceinline__ float4 ld_cluster_f32x4(uint32_t at) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(at)
               : "memory");
  return v;
}

__device__ __forceinline__ void mbar_arrive_cluster(uint32_t bar) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
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
