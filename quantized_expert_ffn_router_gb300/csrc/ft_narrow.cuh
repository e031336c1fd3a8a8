// ft_narrow.cuh -- values of 16, 8 and 4 bits on the device: rows loaded,
// stored and turned into fp32, and the codes and scales that they are quantised
// to.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "ft_common.cuh"
#include "ft_dequant.cuh"

namespace ft {
namespace {

// ----------------------------------------------------------- 16-bit pairs ---
template <bool F16>
__device__ __forceinline__ float2 unpack2(uint32_t w) {
  if (F16) {
    const __half2 h = *reinterpret_cast<const __half2*>(&w);
    return __half22float2(h);
  }
  return make_float2(bf16_lo(w), bf16_hi(w));
}

template <bool F16>
__device__ __forceinline__ uint32_t pack2(float a, float b) {
  if (F16) {
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}

template <bool F16>
__device__ __forceinline__ float load_one(const uint16_t* p) {
  return F16 ? __half2float(__ushort_as_half(*p)) : bf16_val(*p);
}

template <bool F16>
__device__ __forceinline__ void unpack8(const uint4& v, float* f) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 t = unpack2<F16>(w[i]);
    f[2 * i] = t.x;
    f[2 * i + 1] = t.y;
  }
}

template <bool F16>
__device__ __forceinline__ uint4 pack8(const float* f) {
  return make_uint4(pack2<F16>(f[0], f[1]), pack2<F16>(f[2], f[3]), pack2<F16>(f[4], f[5]), pack2<F16>(f[6], f[7]));
}

// 32 bytes to or from two places of 16, in one access where they are one
// 32-byte place: two would each touch half of every sector.
__device__ __forceinline__ void store32(void* p, uint4 a, uint4 b, bool whole) {
  if (whole) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(a.x), "r"(a.y), "r"(a.z),
                 "r"(a.w), "r"(b.x), "r"(b.y), "r"(b.z), "r"(b.w)
                 : "memory");
  } else {
    static_cast<uint4*>(p)[0] = a;
    static_cast<uint4*>(p)[1] = b;
  }
}

__device__ __forceinline__ void load32(const void* p, uint4& a, uint4& b, bool whole) {
  if (whole) {
    asm volatile("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(a.x), "=r"(a.y), "=r"(a.z), "=r"(a.w), "=r"(b.x), "=r"(b.y), "=r"(b.z), "=r"(b.w)
                 : "l"(p));
  } else {
    a = static_cast<const uint4*>(p)[0];
    b = static_cast<const uint4*>(p)[1];
  }
}

// --------------------------------------------------------------- quantising ---
// The smallest e >= kMinExponent with amax <= top * 2^e, where top = 1.t * 2^x
// and t_bits are top's fraction bits: exact, from the bits of amax.
__device__ __forceinline__ int row_exponent(float amax, int x, uint32_t t_bits) {
  const uint32_t b = __float_as_uint(amax);
  const int e = static_cast<int>(b >> 23) - 127 - x + ((b & 0x7fffffu) > t_bits ? 1 : 0);
  return max(e, kMinExponent);
}

__device__ __forceinline__ float pow2f(int e) { return __uint_as_float(static_cast<uint32_t>(e + 127) << 23); }

// Two E4M3 codes, `a` in the low byte; |x| > 448 gives 448, NaN stays NaN.
__device__ __forceinline__ uint32_t to_e4m3x2(float a, float b) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(b), "f"(a));
  return r;
}

// Two E2M1 codes in a byte, `a` in the low nibble.
__device__ __forceinline__ uint32_t to_e2m1x2(float a, float b) {
  uint32_t r;
  asm("{\n .reg .b8 c;\n cvt.rn.satfinite.e2m1x2.f32 c, %1, %2;\n cvt.u32.u8 %0, c;\n}" : "=r"(r) : "f"(b), "f"(a));
  return r;
}

__device__ __forceinline__ float finite_abs(float x) {
  const float a = fabsf(x);
  return a <= 3.4028235e38f ? a : 0.f;
}

// Half a block's E2M1 codes from values that are scaled already.
__device__ __forceinline__ uint32_t codes_e2m1(const float (&z)[8]) {
  uint32_t w = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) w |= to_e2m1x2(z[2 * i], z[2 * i + 1]) << (8 * i);
  return w;
}

__device__ __forceinline__ float e4m3_value(uint32_t code) {
  return __half2float(__ushort_as_half(static_cast<uint16_t>(cvt_e4m3x2(code))));
}

}  // namespace
}  // namespace ft
