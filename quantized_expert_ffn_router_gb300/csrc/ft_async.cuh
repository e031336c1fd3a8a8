// ft_async.cuh -- mbarrier / bulk-copy (TMA) / programmatic-dependent-launch
// helpers written as inline PTX for sm_103a, with bounded waits.
#pragma once

#include <stdint.h>

#include "ft_common.cuh"

namespace ft {

// A bounded wait gives up after this many nanoseconds of the global timer and
// records FT_ERR_TIMEOUT; nothing in this library spins without a limit.
constexpr uint64_t kWaitLimitNs = 2000000000ull;  // 2 s

__device__ __forceinline__ uint32_t smem_u32(const void* p) {
  return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}

__device__ __forceinline__ uint64_t global_timer_ns() {
  uint64_t t;
  asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
  return t;
}

__device__ __forceinline__ void mbar_init(uint64_t* bar, uint32_t count) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(smem_u32(bar)), "r"(count) : "memory");
}

__device__ __forceinline__ void fence_barrier_init() {
  asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
}

__device__ __forceinline__ void mbar_arrive_expect_tx(uint64_t* bar, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(smem_u32(bar)), "r"(bytes)
               : "memory");
}

__device__ __forceinline__ void mbar_arrive(uint64_t* bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_u32(bar)) : "memory");
}

__device__ __forceinline__ bool mbar_try_wait(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n"
      " selp.u32 %0, 1, 0, p;\n}"
      : "=r"(ok)
      : "r"(smem_u32(bar)), "r"(parity)
      : "memory");
  return ok != 0;
}

// What the status word holds now (0 without one).
__device__ __forceinline__ int32_t status_now(const int32_t* status) {
  return status != nullptr ? *reinterpret_cast<const volatile int32_t*>(status) : 0;
}

// Wait for the phase with the given parity; false (and FT_ERR_TIMEOUT
// recorded) if it has not completed within kWaitLimitNs.  OTHERS: false, too,
// as soon as another wait is seen to have given up (for kernels that do not
// look for one before they begin).
template <bool OTHERS = false>
__device__ __forceinline__ bool mbar_wait(uint64_t* bar, uint32_t parity, int32_t* status) {
  if (mbar_try_wait(bar, parity)) return true;
  const uint64_t t0 = global_timer_ns();
  for (uint32_t i = 1;; ++i) {
    if (mbar_try_wait(bar, parity)) return true;
    if (OTHERS && (i & 255u) == 0 && status_now(status) == FT_ERR_TIMEOUT) return false;
    if ((i & 255u) == 0 && global_timer_ns() - t0 > kWaitLimitNs) {
      record_status(status, FT_ERR_TIMEOUT);
      return false;
    }
  }
}

// mbar_wait by every lane of a warp with one verdict for the whole warp (a
// lane that gave up makes every lane give up), for warps that run
// warp-collective instructions (tcgen05.ld) after the wait.
template <bool OTHERS = false>
__device__ __forceinline__ bool mbar_wait_warp(uint64_t* bar, uint32_t parity, int32_t* status) {
  return __all_sync(0xffffffffu, mbar_wait<OTHERS>(bar, parity, status));
}

// True (for the whole CTA) when an earlier wait of this stream's work already
// gave up: kernels with bounded waits then return at once instead of waiting
// out their own.  Every thread of the CTA must call it (it holds a barrier).
__device__ __forceinline__ bool prior_timeout(const int32_t* status) {
  __shared__ int s_skip;
  if (threadIdx.x == 0)
    s_skip = status != nullptr && *reinterpret_cast<const volatile int32_t*>(status) == FT_ERR_TIMEOUT;
  __syncthreads();
  return s_skip != 0;
}

// Bulk copy global -> shared (no tensor map), completion counted on `bar`.
// Addresses 16-byte aligned, size a multiple of 16.
__device__ __forceinline__ void bulk_g2s(void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
          smem_u32(dst)),
      "l"(src), "r"(bytes), "r"(smem_u32(bar))
      : "memory");
}

// Bulk prefetch of global memory into L2 (no destination, no completion).
// Address 16-byte aligned, size a multiple of 16.
__device__ __forceinline__ void l2_prefetch(const void* src, uint32_t bytes) {
  asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(src), "r"(bytes) : "memory");
}

// GPU-scope acquire load / release store / acquire-release wrapping increment
// of a 32-bit word in global memory, and the proxy fence that orders plain
// stores before later bulk-copy (async proxy) reads of the same bytes.
__device__ __forceinline__ uint32_t ld_acquire_gpu(const uint32_t* p) {
  uint32_t v;
  asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
  return v;
}
__device__ __forceinline__ void st_release_gpu(uint32_t* p, uint32_t v) {
  asm volatile("st.release.gpu.global.u32 [%0], %1;" ::"l"(p), "r"(v) : "memory");
}
// old = *p; *p = (old >= limit) ? 0 : old + 1; returns old.
__device__ __forceinline__ uint32_t atom_inc_acq_rel_gpu(uint32_t* p, uint32_t limit) {
  uint32_t old;
  asm volatile("atom.acq_rel.gpu.global.inc.u32 %0, [%1], %2;" : "=r"(old) : "l"(p), "r"(limit) : "memory");
  return old;
}
__device__ __forceinline__ void fence_proxy_async_global() {
  asm volatile("fence.proxy.async.global;" ::: "memory");
}

// Programmatic dependent launch: let the next grid in the stream start, and
// wait for the previous grid's completion and memory.
__device__ __forceinline__ void pdl_launch_dependents() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}
__device__ __forceinline__ void pdl_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// A launch whose grid may start while the one before it on the stream drains;
// the kernel waits (pdl_wait) before it touches memory.
template <typename Kernel, typename Args>
ft_status launch_pdl(Kernel kernel, dim3 grid, int block, size_t smem, cudaStream_t s, const Args& a, const char* what) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(block);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  cudaLaunchKernelEx(&cfg, kernel, a);
  return launch_check(what);
}

}  // namespace ft
