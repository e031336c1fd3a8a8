// kv.cu -- rotary positions, and the paged key-value cache's rows written
// (rotated and quantised on the way) and read back.
//
// Both kernels stream: every value is read once and written once, so
// they are bound by HBM (or, for one token, by the launch and one chain of
// dependent loads).  A head row is spread over the lanes of part of one warp,
// 16 elements a lane, so that a row's maximum is a few shuffles and every
// access is a 16- or 32-byte one.
//
// What they measured (GPU time in a graph, inputs beyond L2; of 6.70 TB/s):
//   4099 tokens x 40 heads of 128 rotated, half of each head: 15.6 us (80%), 20000 tokens 66.7 us (92%);
//   8192 tokens, 32 + 2 x 8 heads of 128, rotated, into E4M3: 35.4 us (78%), 20000 tokens 81.2 us (83%);
//   the same into bf16: 35.1 us (86%), 80.7 us (91%);
//   20000 tokens, 16 + 2 x 2 heads of 128, rotated, into NVFP4: 54.3 us (52%);
//   16384 tokens x 2 x 8 heads of 128 read back as bf16: E4M3 18.4 us (82%), bf16 22.4 (89%), NVFP4 17.5 (74%).
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <math.h>

#include "ft_kv.cuh"

namespace ft {
namespace {

// ------------------------------------------------------------------ angles ---
// cos(2 pi j / 128), j = 0..32, each as the sum of two floats.
__device__ const float2 kCosine[33] = {
    {0x1.000000p+0f, 0x0.0p+0f}, {0x1.ff621ep-1f, 0x1.bcb6c0p-28f},
    {0x1.fd88dap-1f, 0x1.e89294p-28f}, {0x1.fa7558p-1f, -0x1.eeb5d2p-30f},
    {0x1.f6297cp-1f, 0x1.feeb96p-26f}, {0x1.f0a7f0p-1f, -0x1.1b73cap-27f},
    {0x1.e9f416p-1f, -0x1.273a44p-26f}, {0x1.e21210p-1f, 0x1.3da1bap-27f},
    {0x1.d906bcp-1f, 0x1.e651a8p-26f}, {0x1.ced7b0p-1f, -0x1.786712p-26f},
    {0x1.c38b30p-1f, -0x1.cfe84ap-26f}, {0x1.b72834p-1f, 0x1.465b90p-27f},
    {0x1.a9b662p-1f, 0x1.21d434p-26f}, {0x1.9b3e04p-1f, 0x1.fce1d0p-27f},
    {0x1.8bc806p-1f, 0x1.62a2e8p-26f}, {0x1.7b5df2p-1f, 0x1.3557d8p-28f},
    {0x1.6a09e6p-1f, 0x1.9fcef4p-27f}, {0x1.57d694p-1f, -0x1.6e626cp-26f},
    {0x1.44cf32p-1f, 0x1.424776p-27f}, {0x1.30ff80p-1f, -0x1.8f47e4p-28f},
    {0x1.1c73b4p-1f, -0x1.9465cep-27f}, {0x1.07387ap-1f, -0x1.b74004p-27f},
    {0x1.e2b5d4p-2f, -0x1.fe4270p-28f}, {0x1.b5d100p-2f, 0x1.3c2b98p-27f},
    {0x1.87de2ap-2f, 0x1.abaa58p-28f}, {0x1.58f9a8p-2f, -0x1.4a9c04p-27f},
    {0x1.294062p-2f, 0x1.dab3e0p-27f}, {0x1.f19f98p-3f, -0x1.37a838p-29f},
    {0x1.8f8b84p-3f, -0x1.cb2cfap-30f}, {0x1.2c8106p-3f, 0x1.d1cc28p-28f},
    {0x1.917a6cp-4f, -0x1.eb25e4p-31f}, {0x1.91f660p-5f, -0x1.de44fcp-30f},
    {0x0.0p+0f, 0x0.0p+0f}};

// hi + lo of a + b, exactly (Knuth).
__device__ __forceinline__ float2 two_sum(float a, float b) {
  const float s = __fadd_rn(a, b);
  const float bb = __fsub_rn(s, a);
  return make_float2(s, __fadd_rn(__fsub_rn(a, __fsub_rn(s, bb)), __fsub_rn(b, bb)));
}

// cos and sin of a * 2^-64 turns, times m, in fp32: (cos, sin).
__device__ __forceinline__ float2 turn_f32(int64_t a, float m) {
  float s, c;
  sincospif(static_cast<float>(static_cast<int32_t>(a >> 32)) * 0x1p-31f, &s, &c);
  return make_float2(c * m, s * m);
}

// The same to about 2^-34, as pairs of floats: *hi = (cos, sin), *lo the rest.
// The angle is the nearest of 128 steps of the circle (from the table) plus a
// remainder d of at most 2^-8 turn (0.0246): cos d - 1 and sin d by their
// series, joined by the addition theorem in two-float arithmetic.  The
// rounding-mode intrinsics keep the compiler from fusing the error terms away.
__device__ __forceinline__ void turn_pair(int64_t a, float m, float2* hi, float2* lo) {
  const int64_t step = (a + (int64_t(1) << 56)) >> 57;
  const int64_t r = a - (step << 57);
  const int j = static_cast<int>(step) & 127, i = j & 31;
  const float2 u = kCosine[i], w = kCosine[32 - i];
  float2 C = (j & 32) ? w : u, S = (j & 32) ? u : w;
  if (((j + 32) & 64) != 0) C = make_float2(-C.x, -C.y);
  if ((j & 64) != 0) S = make_float2(-S.x, -S.y);
  // d = 2 pi r 2^-64
  const float k_hi = 0x1.921fb6p-62f, k_lo = -0x1.777a5cp-87f;
  const float rh = static_cast<float>(r);
  const float rl = static_cast<float>(r - static_cast<int64_t>(rh));
  const float d = __fmul_rn(rh, k_hi);
  const float dl = __fmaf_rn(rh, k_hi, -d) + (rh * k_lo + rl * k_hi);
  const float d2 = d * d;
  const float c1 = d2 * (-0.5f + d2 * (1.f / 24 - d2 * (1.f / 720))) - d * dl;   // cos d - 1
  const float sl = dl + d * d2 * (-1.f / 6 + d2 * (1.f / 120));                  // sin d - d
  // cos = C + C c1 - S sin d, sin = S + S c1 + C sin d
  float2 out_c, out_s;
  {
    const float p = __fmul_rn(S.x, d);
    const float pe = __fmaf_rn(S.x, d, -p) + (S.x * sl + S.y * d);
    const float2 t = two_sum(C.x, -p);
    out_c = two_sum(t.x, t.y + (C.x * c1 - pe) + C.y);
  }
  {
    const float p = __fmul_rn(C.x, d);
    const float pe = __fmaf_rn(C.x, d, -p) + (C.x * sl + C.y * d);
    const float2 t = two_sum(S.x, p);
    out_s = two_sum(t.x, t.y + (S.x * c1 + pe) + S.y);
  }
  const float cm = __fmul_rn(out_c.x, m), sm = __fmul_rn(out_s.x, m);
  *hi = make_float2(cm, sm);
  *lo = make_float2(__fmaf_rn(out_c.x, m, -cm) + out_c.y * m, __fmaf_rn(out_s.x, m, -sm) + out_s.y * m);
}

// x c - y s from two-float c and s, rounded to odd: the last bit is set
// wherever the sum is not exactly a float, so that rounding it again to the
// few bits of a code rounds the sum itself, ties included.
__device__ __forceinline__ float rotate_odd(float x, float y, float c, float cl, float s, float sl) {
  const float p = __fmul_rn(x, c), q = __fmul_rn(y, s);
  const float pe = __fmaf_rn(x, c, -p), qe = __fmaf_rn(y, s, -q);
  const float2 t = two_sum(p, -q);
  if (!(fabsf(t.x) <= 3.4028235e38f)) return t.x;  // infinite or NaN
  const float rest = t.y + (pe - qe) + (x * cl - y * sl);
  const float2 h = two_sum(t.x, rest);
  uint32_t b = __float_as_uint(h.x);
  if (h.y != 0.f) {
    if ((h.y < 0.f) != (h.x < 0.f)) b -= 1;
    b |= 1;
  }
  return __uint_as_float(b);
}

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

// ------------------------------------------------------------ rotate, write ---
enum { kPairs, kHalves, kAny };
constexpr int kMaxBatch = 16;
struct WriteArgs {
  KvView kv;
  const uint16_t* in[3];  // q, k, v
  int64_t in_tok[3], in_head[3];
  uint16_t* q_out;
  int64_t out_tok, out_head;
  const int32_t* pos;       // places in the cache (NULL: rotation only)
  const int32_t* rope_pos;  // positions of the rotation
  const int64_t* freqs;
  float mscale;
  int32_t rot, half;        // rotated channels, half of them; 0: no rotation
  int32_t T, Hq, Hkv, D;
  int32_t lanes_log2;       // lanes of one row
  int32_t parts;            // CTAs of one token
  int32_t batch;            // tokens of a CTA
  int32_t wide_in, wide_out;  // inputs, q_out: every 16 channels are a 32-byte place
  int32_t* status;
};

// Where frequency f's cosine (or sine) lies among `half`: 16-byte chunks in an
// order that lets 8 lanes read every other chunk without a bank conflict.
__device__ __forceinline__ int turn_at(int f) {
  const int j = f >> 2;
  return ((j ^ ((j >> 3) & 1)) << 2) | (f & 3);
}

// One lane's 16 channels of one row, as loaded: two chunks of 8, and the other
// sides of their rotations where the lane does not hold them (kAny).
template <int LAY>
struct Chunks {
  uint4 own[2];
  uint4 other[LAY == kAny ? 2 : 1];
};

// x[16] as E4M3 codes, given the row's exponent.
__device__ __forceinline__ uint4 codes_e4m3(const float (&x)[16], int e) {
  const float inv = pow2f(-e);
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    w[i] = to_e4m3x2(x[4 * i] * inv, x[4 * i + 1] * inv) | (to_e4m3x2(x[4 * i + 2] * inv, x[4 * i + 3] * inv) << 16);
  return make_uint4(w[0], w[1], w[2], w[3]);
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

// The largest finite magnitude of x[16].
__device__ __forceinline__ float largest(const float (&x)[16]) {
  float m = 0.f;
#pragma unroll
  for (int i = 0; i < 16; ++i) m = fmaxf(m, fabsf(x[i]));  // NaN is passed over
  if (m > 3.4028235e38f) {
    m = 0.f;
#pragma unroll
    for (int i = 0; i < 16; ++i) m = fmaxf(m, finite_abs(x[i]));
  }
  return m;
}

// A CTA takes (a part of the rows of) `batch` tokens, one after the other,
// loading the next rows while it works on these.  Before the first, its
// threads share out the work of looking up the tokens' rows in the cache and
// of the tokens' rot/2 cosines and sines, which all heads use.
//
// A lane holds two chunks of 8 channels.
//   kPairs   neighbouring chunks; interleaved rotations (or none) stay inside.
//   kHalves  chunks c and c + half / 8, the two sides of the same 8 rotations
//            (half layout, halves of whole chunks; NVFP4: of whole blocks,
//            which two neighbouring lanes then share).
//   kAny     neighbouring chunks, half layout: the other side is loaded as
//            well (it is in L1, another lane's own).
//
// FMT: a cache format, or -1 to rotate q only.
//
// Rotated keys that are quantised.  A code has to be that of the exact
// rotation, but fp32 is good to d = 2^-20.5 (|u| + |v|) m of it (angle 2^-24
// turn and sincospif 2 ulp: 2^-21.8; two products and a sum: 2^-22.4).  So both
// ends x - d and x + d are quantised: where they agree, that is the code;
// where a border lies between (about one element in 2^16), its lane rotates it
// again in two-float arithmetic.
template <bool F16, int FMT, int LAY>
__global__ void __launch_bounds__(512, LAY == kAny ? 1 : 2) write_kernel(const __grid_constant__ WriteArgs a) {
  constexpr bool kQuant = FMT == FT_KV_E4M3 || FMT == FT_KV_NVFP4;
  extern __shared__ __align__(16) float turns[];  // [batch][cosines, sines][half, rounded up to whole chunk pairs]
  __shared__ uint32_t rows_s[kMaxBatch];          // head 0's row of each token's place
  const int half_up = (a.half + 31) & ~31;
  const uint32_t group = blockIdx.x / a.parts, part = blockIdx.x - group * a.parts;
  const int t0 = group * a.batch, tokens = min(a.batch, a.T - t0);
  const int lanes = 1 << a.lanes_log2;
  const int rows = a.Hq + (FMT >= 0 ? 2 * a.Hkv : 0);
  const int step = (a.parts * blockDim.x) >> a.lanes_log2;
  const int l = threadIdx.x & (lanes - 1);
  const int hc = a.half >> 3;
  int c0, c1;  // the lane's chunks
  if (LAY == kHalves && l < hc) {
    c0 = l;
    c1 = l + hc;
  } else {
    c0 = 2 * l;
    c1 = 2 * l + 1;
  }
  const bool has0 = c0 * 8 < a.D, has1 = c1 * 8 < a.D;
  const bool vec = (a.half & 7) == 0;
  const int r_cta = (part * blockDim.x) >> a.lanes_log2;
  const int rounds = (rows - r_cta + step - 1) / step;  // the same for every thread of the CTA

  // Of the next token's turn: the row, what it is, and where its channels are.
  // Lanes past the last row, or past the last channel, load others again: valid
  // reads, whose results are not stored.  4-bit keys and values take so much
  // longer than queries that the warps change places from token to token (20000
  // tokens, 16 + 2 x 2 heads of 128: 63.8 us, then 54.9; 8-bit rows, 32 + 2 x 8
  // heads: 80.2, then 84.2).
  constexpr bool kMoves = FMT == FT_KV_NVFP4;
  const int warps = blockDim.x >> 5, sub = (threadIdx.x & 31) >> a.lanes_log2, of_warp_log2 = 5 - a.lanes_log2;
  int place = threadIdx.x >> 5;  // the warp's place among the CTA's at this token
  int next_kind, next_h;
  bool next_live;
  const uint16_t* next_src;
  const auto turn_to = [&](int round, int tk) {
    const int row = r_cta + round * step + (place << of_warp_log2) + sub, r = min(row, rows - 1);
    next_live = row < rows;
    next_kind = r < a.Hq ? 0 : r < a.Hq + a.Hkv ? 1 : 2;
    next_h = next_kind == 0 ? r : next_kind == 1 ? r - a.Hq : r - a.Hq - a.Hkv;
    next_src = a.in[next_kind] + static_cast<int64_t>(t0 + tk) * a.in_tok[next_kind] + next_h * a.in_head[next_kind];
  };
  const int l0 = has0 ? c0 * 8 : 0, l1 = has1 ? c1 * 8 : 0;
  const int o0 = has0 && c0 < 2 * hc ? (c0 < hc ? c0 + hc : c0 - hc) * 8 : 0;  // the other sides
  const int o1 = has1 && c1 < 2 * hc ? (c1 < hc ? c1 + hc : c1 - hc) * 8 : 0;
  const auto load = [&](const uint16_t* from, Chunks<LAY>& c) {
    if (LAY != kHalves && a.wide_in) {
      load32(from + l0, c.own[0], c.own[1], true);
    } else {
      c.own[0] = *reinterpret_cast<const uint4*>(from + l0);
      c.own[1] = *reinterpret_cast<const uint4*>(from + l1);
    }
    if constexpr (LAY == kAny) {
      c.other[0] = c.other[1] = make_uint4(0, 0, 0, 0);
      if (vec) {
        c.other[0] = *reinterpret_cast<const uint4*>(from + o0);
        c.other[1] = *reinterpret_cast<const uint4*>(from + o1);
      }
    }
  };

  pdl_wait();
  Chunks<LAY> next;
  turn_to(0, 0);
  load(next_src, next);

  if (FMT >= 0 && threadIdx.x < tokens) {
    const int32_t place = a.pos[t0 + threadIdx.x];
    rows_s[threadIdx.x] = place < 0 ? kNoRow : kv_token_row(a.kv, kv_seq(a.kv, t0 + threadIdx.x), place, a.status);
  }
  if (a.rot > 0) {
    for (int i = threadIdx.x; i < tokens * a.half; i += blockDim.x) {
      const int token = i / a.half, f = i - token * a.half;
      const int64_t p = a.rope_pos[t0 + token];
      const float2 cs = turn_f32(static_cast<int64_t>(static_cast<uint64_t>(p) * static_cast<uint64_t>(a.freqs[f])), a.mscale);
      turns[token * 2 * half_up + turn_at(f)] = cs.x;
      turns[token * 2 * half_up + half_up + turn_at(f)] = cs.y;
    }
  }
  __syncthreads();

  // kAny: the other sides of the lane's rotations
  const auto other_sides = [&](const Chunks<LAY>& c, const uint16_t* from, float (&y)[16]) {
    if (vec) {
      unpack8<F16>(c.other[0], y);
      unpack8<F16>(c.other[LAY == kAny ? 1 : 0], y + 8);  // of lanes without rotated channels: not used
    } else {
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const int ch = (i < 8 ? c0 : c1) * 8 + (i & 7);
        y[i] = ch < a.rot ? load_one<F16>(from + (ch < a.half ? ch + a.half : ch - a.half)) : 0.f;
      }
    }
  };
  // What fp32's rotation of the lane's channels may be off by: 2^-20.5 (|u| +
  // |v|) m; that is at most 2^-20 (|x| + |y|) of the rotated pair.  Nothing for
  // values, infinite ones too.
  const auto uncertainty = [&](const Chunks<LAY>& c, const uint16_t* from, bool any, const float (&x)[16], float (&d)[16]) {
    if (LAY == kAny) {
      const float off = 6.7434956e-7f * fabsf(a.mscale);
      float u[16], y[16];
      unpack8<F16>(c.own[0], u);
      unpack8<F16>(c.own[1], u + 8);
      other_sides(c, from, y);
#pragma unroll
      for (int i = 0; i < 16; ++i) d[i] = any && (i < 8 ? c0 : c1) * 8 + (i & 7) < a.rot ? (fabsf(u[i]) + fabsf(y[i])) * off : 0.f;
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int iu = LAY == kPairs ? 2 * i : i, iv = LAY == kPairs ? 2 * i + 1 : i + 8;
        const bool turns_too = any && (LAY == kPairs ? 8 * l + i < a.half : l < hc);
        d[iu] = d[iv] = turns_too ? (fabsf(x[iu]) + fabsf(x[iv])) * 0x1p-20f : 0.f;
      }
    }
  };

  const int f0 = LAY == kPairs ? 8 * l : 8 * c0;  // the lane's first frequency, and how many it turns by
  const int turning = LAY == kPairs ? min(8, a.half - f0) : l < hc ? 8 : 0;
  const int turn0 = turn_at(f0), turn1 = turn_at(f0 + 4);
  const bool filled = a.D == (16 << a.lanes_log2);  // every lane has its channels

  for (int round = 0; round < rounds; ++round) {
#pragma unroll 1
    for (int tk = 0; tk < tokens; ++tk) {
      const int kind = next_kind, h = next_h, w = kind == 2 ? 1 : 0;
      const bool live = next_live, spin = a.rot > 0 && kind < 2, exact = kQuant && kind == 1 && spin;
      const uint16_t* src = next_src;
      const float* cosines = turns + tk * 2 * half_up;
      const float* sines = cosines + half_up;
      float x[16];
      unpack8<F16>(next.own[0], x);
      unpack8<F16>(next.own[1], x + 8);
      Chunks<LAY> now;  // kAny: the other sides are still to be read
      if (LAY == kAny) now = next;
      if (tk + 1 < tokens || round + 1 < rounds) {
        if (kMoves) place = place + 1 == warps ? 0 : place + 1;
        if (kMoves || tk + 1 == tokens)
          turn_to(tk + 1 < tokens ? round : round + 1, tk + 1 < tokens ? tk + 1 : 0);
        else
          next_src += a.in_tok[kind];
        load(next_src, next);
      }
      if (spin) {
        if (LAY == kPairs || LAY == kHalves) {
          // 8 rotations: channels (2i, 2i + 1), or (i, i + 8)
          if (turning > 0) {
            float cs[8], sn[8];
#pragma unroll
            for (int i = 0; i < 8; i += 4) {
              *reinterpret_cast<float4*>(cs + i) = *reinterpret_cast<const float4*>(cosines + (i ? turn1 : turn0));
              *reinterpret_cast<float4*>(sn + i) = *reinterpret_cast<const float4*>(sines + (i ? turn1 : turn0));
            }
            const auto spin_one = [&](int i) {
              const int iu = LAY == kPairs ? 2 * i : i, iv = LAY == kPairs ? 2 * i + 1 : i + 8;
              const float u = x[iu], v = x[iv];
              x[iu] = u * cs[i] - v * sn[i];
              x[iv] = v * cs[i] + u * sn[i];
            };
            if (LAY == kHalves || vec) {
#pragma unroll
              for (int i = 0; i < 8; ++i) spin_one(i);
            } else {  // the last of the rotated channels
#pragma unroll
              for (int i = 0; i < 8; ++i)
                if (i < turning) spin_one(i);
            }
          }
        } else {
          float y[16];
          other_sides(now, src, y);
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const int c = (i < 8 ? c0 : c1) * 8 + (i & 7);
            if (c < a.rot) {
              const bool left = c < a.half;
              const int at = turn_at(left ? c : c - a.half);
              x[i] = x[i] * cosines[at] - (left ? y[i] : -y[i]) * sines[at];
            }
          }
        }
      }
      __syncwarp();  // in place: the row's lanes have loaded both sides before any of them stores
      if (kind == 0 || FMT < 0) {
        uint16_t* dst_q = a.q_out + static_cast<int64_t>(t0 + tk) * a.out_tok + h * a.out_head;
        if (LAY != kHalves && live && has1) {
          store32(dst_q + c0 * 8, pack8<F16>(x), pack8<F16>(x + 8), a.wide_out != 0);
        } else {
          if (live && has0) *reinterpret_cast<uint4*>(dst_q + c0 * 8) = pack8<F16>(x);
          if (live && has1) *reinterpret_cast<uint4*>(dst_q + c1 * 8) = pack8<F16>(x + 8);
        }
      }
      if (FMT < 0 || __all_sync(0xffffffffu, kind == 0)) continue;
      const uint32_t row0 = rows_s[tk];
      const bool put = live && kind > 0 && row0 != kNoRow;
      if (!__any_sync(0xffffffffu, put)) continue;
      const uint32_t row = row0 + static_cast<uint32_t>(h) * a.kv.at.head_stride;
      uint8_t* dst = a.kv.data[w] + static_cast<uint64_t>(row) * a.kv.row_bytes;
      if (!kQuant) {
        if (put && has0) *reinterpret_cast<uint4*>(dst + c0 * 16) = pack8<F16>(x);
        if (put && has1) *reinterpret_cast<uint4*>(dst + c1 * 16) = pack8<F16>(x + 8);
        continue;
      }
      constexpr int top = FMT == FT_KV_E4M3 ? 8 : 11;                           // 448 = 1.75 * 2^8,
      constexpr uint32_t top_bits = FMT == FT_KV_E4M3 ? 0x600000u : 0x280000u;  // 2688 = 1.3125 * 2^11
      const auto row_largest = [&](float m) {
        for (int o = lanes >> 1; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
        return m;
      };
      if (!filled) {
#pragma unroll
        for (int i = 0; i < 16; ++i) x[i] = (i < 8 ? has0 : has1) ? x[i] : 0.f;
      }
      // What the exact rotation of the elements in `unsure` (a bit each) gives.
      const auto rotate_again = [&](uint32_t unsure) {
        const int64_t p = a.rope_pos[t0 + tk];
        while (unsure != 0) {
          const int i = __ffs(unsure) - 1;
          unsure &= unsure - 1;
          const int c = (i < 8 ? c0 : c1) * 8 + (i & 7);
          if (c >= a.rot) continue;
          const bool left = LAY == kPairs ? (c & 1) == 0 : c < a.half;
          const int f = LAY == kPairs ? c >> 1 : left ? c : c - a.half;
          const int o = LAY == kPairs ? c ^ 1 : left ? c + a.half : c - a.half;
          float2 hi, lo;
          turn_pair(static_cast<int64_t>(static_cast<uint64_t>(p) * static_cast<uint64_t>(a.freqs[f])), a.mscale, &hi, &lo);
          const float u = load_one<F16>(src + c), v = load_one<F16>(src + o);
          const float y = rotate_odd(u, left ? v : -v, hi.x, lo.x, hi.y, lo.y);
#pragma unroll
          for (int j = 0; j < 16; ++j) x[j] = j == i ? y : x[j];
        }
        __syncwarp();
      };
      int e;
      if constexpr (FMT == FT_KV_E4M3) {
        float amax = row_largest(largest(x));
        e = row_exponent(amax, top, top_bits);
        uint4 code;
        if (!__any_sync(0xffffffffu, exact)) {
          code = codes_e4m3(x, e);
        } else {
          // Both ends; the row's largest is at least the largest pair's size /
          // sqrt 2, so off by at most 2^-19 of itself.
          float d[16], z[16];
          uncertainty(now, src, exact, x, d);
#pragma unroll
          for (int i = 0; i < 16; ++i) z[i] = x[i] - d[i];
          code = codes_e4m3(z, e);
#pragma unroll
          for (int i = 0; i < 16; ++i) z[i] = x[i] + d[i];
          const uint4 up = codes_e4m3(z, e);
          const float part = amax * 0x1p-19f;
          const bool all = row_exponent(amax - part, top, top_bits) != row_exponent(amax + part, top, top_bits);
          const uint32_t differ[4] = {code.x ^ up.x, code.y ^ up.y, code.z ^ up.z, code.w ^ up.w};
          if (__any_sync(0xffffffffu, exact && live && (all || (differ[0] | differ[1] | differ[2] | differ[3]) != 0))) {
            uint32_t unsure = all ? 0xffffu : 0;
#pragma unroll
            for (int i = 0; i < 16; ++i)
              if ((differ[i >> 2] >> (8 * (i & 3))) & 0xff) unsure |= 1u << i;
            rotate_again(exact && live ? unsure : 0);
            amax = row_largest(largest(x));
            e = row_exponent(amax, top, top_bits);
            code = codes_e4m3(x, e);
          }
        }
        if (put && has0) *reinterpret_cast<uint2*>(dst + c0 * 8) = make_uint2(code.x, code.y);
        if (put && has1) *reinterpret_cast<uint2*>(dst + c1 * 8) = make_uint2(code.z, code.w);
      } else {
        constexpr bool kShared = LAY == kHalves;  // a rotated channel's block is half this lane's, half its neighbour's
        const bool shared = kShared && l < hc;
        // of the lane's two chunks, to that of the blocks they are in
        const auto join = [&](float (&m)[2]) {
          const float both = fmaxf(m[0], m[1]);
          if (kShared) {
            const float n0 = __shfl_xor_sync(0xffffffffu, m[0], 1), n1 = __shfl_xor_sync(0xffffffffu, m[1], 1);
            m[0] = shared ? fmaxf(m[0], n0) : both;
            m[1] = shared ? fmaxf(m[1], n1) : both;
          } else {
            m[0] = m[1] = both;
          }
        };
        // Codes without divisions: a product with 1 / block scale is good to
        // 2^-21, which widens d, and values are then treated as keys are (the
        // divisions of both ends took twice the time).
        float d[16], m[2] = {0.f, 0.f}, far[2] = {0.f, 0.f};
        bool odd = false;  // infinities and NaN
        if (__any_sync(0xffffffffu, exact)) {
          uncertainty(now, src, exact, x, d);
        } else {
#pragma unroll
          for (int i = 0; i < 16; ++i) d[i] = 0.f;
        }
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const float size = fabsf(x[i]);
          d[i] = fmaf(size, 0x1p-21f, d[i]);
          m[i >> 3] = fmaxf(m[i >> 3], size);
          far[i >> 3] = fmaxf(far[i >> 3], d[i]);
          odd |= !(size <= 3.4028235e38f);
        }
        join(m);
        join(far);
        const float amax = row_largest(fmaxf(m[0], m[1])), part = amax * 0x1p-19f;
        e = row_exponent(amax, top, top_bits);
        const float inv = pow2f(-e);
        // An infinity anywhere in a rotated row leaves all of its lanes in doubt: amax - part is NaN there, whose
        // exponent is one more than infinity's.
        bool all = odd || (exact && row_exponent(amax - part, top, top_bits) != row_exponent(amax + part, top, top_bits));
        uint32_t code[2], differ[2], block[2];
        float per = 0.f;
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          if (c == 0 || kShared) {
            const uint32_t ends = to_e4m3x2((m[c] + far[c]) * (inv * (1.f / 6.f)), (m[c] - far[c]) * (inv * (1.f / 6.f)));
            block[c] = ends & 0xffu;
            all |= block[c] != ends >> 8;
            const float bs = e4m3_value(block[c]);
            per = bs > 0.f ? __fdividef(inv, bs) : 0.f;
          } else {
            block[c] = block[0];
          }
          float low[8], high[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            low[i] = (x[8 * c + i] - d[8 * c + i]) * per;
            high[i] = (x[8 * c + i] + d[8 * c + i]) * per;
          }
          code[c] = per > 0.f ? codes_e2m1(low) : 0;
          differ[c] = per > 0.f ? code[c] ^ codes_e2m1(high) : 0;
        }
        if (__any_sync(0xffffffffu, put && (all || (differ[0] | differ[1]) != 0))) {
          uint32_t unsure = all ? 0xffffu : 0;
#pragma unroll
          for (int i = 0; i < 16; ++i)
            if ((differ[i >> 3] >> (4 * (i & 7))) & 0xf) unsure |= 1u << i;
          rotate_again(exact && live ? unsure : 0);
          float nan[2] = {0.f, 0.f};
          m[0] = m[1] = 0.f;
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            m[i >> 3] = fmaxf(m[i >> 3], finite_abs(x[i]));
            nan[i >> 3] = isnan(x[i]) ? 1.f : nan[i >> 3];
          }
          join(m);
          join(nan);
          e = row_exponent(row_largest(fmaxf(m[0], m[1])), top, top_bits);
          const float scale = pow2f(-e);
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            block[c] = to_e4m3x2(nan[c] > 0.f ? NAN : m[c] * scale / 6.f, 0.f) & 0xffu;
            const float bs = e4m3_value(block[c]);
            float z[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) z[i] = x[8 * c + i] * scale / bs;
            code[c] = bs > 0.f ? codes_e2m1(z) : 0;
          }
        }
        if (kShared) {
          if (put && has0) *reinterpret_cast<uint32_t*>(dst + c0 * 4) = code[0];
          if (put && has1) *reinterpret_cast<uint32_t*>(dst + c1 * 4) = code[1];
        } else if (put && has0) {
          *reinterpret_cast<uint2*>(dst + l * 8) = make_uint2(code[0], code[1]);
        }
        // of two lanes that share two blocks, each stores one scale
        const bool second = shared && (l & 1);
        if (put && (second ? has1 : has0))
          a.kv.block[w][static_cast<uint64_t>(row) * (a.D / 16) + ((second ? c1 : c0) >> 1)] =
              static_cast<uint8_t>(second ? block[1] : block[0]);
      }
      if (put && l == 0) a.kv.scale[w][row] = static_cast<uint8_t>(e + 127);
    }
  }
}

// ---------------------------------------------------------------- read back ---
struct ReadArgs {
  KvView kv;
  const int32_t* pos;
  void* out[2];
  int64_t tok[2], head[2];
  FastDiv by_heads;
  uint32_t rows;  // T * Hkv
  int32_t lanes_log2;
  int32_t wide_in, wide_out;  // 16-bit rows of the cache, of the outputs: every 16 elements are a 32-byte place
  int32_t* status;
};

// A lane reads 16 elements of a (token, head)'s key row and of its value row
// (they share the place in the cache, so the dependent loads of position, page
// and row are paid once for both) and writes them out dense.  One such pair a
// lane: with two or four the SMs hold fewer (16384 tokens x 8 heads of 128,
// E4M3 to bf16: 21.2 us, 23.3 and 28.1).
template <int FMT, int DT>
__global__ void __launch_bounds__(256) read_kernel(const __grid_constant__ ReadArgs a) {
  constexpr int W = FMT == FT_KV_NVFP4 ? 2 : FMT == FT_KV_E4M3 ? 4 : 8;  // words of 16 elements
  const int l = threadIdx.x & ((1 << a.lanes_log2) - 1);
  // the launch has up to 2^35 threads, of up to 2^31 rows
  const uint32_t at = static_cast<uint32_t>((uint64_t{blockIdx.x} * 256 + threadIdx.x) >> a.lanes_log2);
  pdl_wait();
  if (at >= a.rows || l * 16 >= a.kv.D) return;
  const uint32_t token = fast_div(at, a.by_heads), head = at - token * a.kv.Hkv;
  const int32_t pos = a.pos[token];
  uint32_t row = kNoRow;
  if (pos >= 0) row = kv_token_row(a.kv, kv_seq(a.kv, token), pos, l == 0 ? a.status : nullptr);
  uint32_t w[2][W], b[2], e[2];
#pragma unroll
  for (int j = 0; j < 2; ++j) {
#pragma unroll
    for (int i = 0; i < W; ++i) w[j][i] = 0;
    b[j] = 0;
    e[j] = 127;
    if (row == kNoRow || a.out[j] == nullptr) continue;
    const uint64_t r = row + head * a.kv.at.head_stride;
    const uint8_t* src = a.kv.data[j] + r * a.kv.row_bytes + l * (W * 4);
    if constexpr (W == 2) {
      const uint2 v = *reinterpret_cast<const uint2*>(src);
      w[j][0] = v.x, w[j][1] = v.y;
      b[j] = a.kv.block[j][r * (a.kv.D / 16) + l];
    } else {
      uint4 v, u;
      if constexpr (W == 8)
        load32(src, v, u, a.wide_in != 0);
      else
        v = *reinterpret_cast<const uint4*>(src);
      w[j][0] = v.x, w[j][1] = v.y, w[j][2] = v.z, w[j][3] = v.w;
      if constexpr (W == 8) w[j][4] = u.x, w[j][5] = u.y, w[j][6] = u.z, w[j][7] = u.w;
    }
    if (W < 8) e[j] = a.kv.scale[j][r];
  }
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    if (a.out[j] == nullptr) continue;
    float x[16];
    if constexpr (W == 8) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float2 v = unpack2<FMT == FT_KV_F16>(w[j][i]);
        x[2 * i] = v.x;
        x[2 * i + 1] = v.y;
      }
    } else {
      uint32_t f[8];  // f16 pairs; code * block scale is exact in fp32
      // held here, not where it is read: the values' loads must not wait for the keys' (0.3 us of one token's read)
      float scale = pow2f(static_cast<int>(held_exponent<FMT>(e[j])) - 127);
      if constexpr (W == 4) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          f[2 * i] = cvt_e4m3x2(w[j][i]);
          f[2 * i + 1] = cvt_e4m3x2(w[j][i] >> 16);
        }
      } else {
        e2m1x8(w[j][0], f);
        e2m1x8(w[j][1], f + 4);
        scale *= unpack2<true>(cvt_e4m3x2(b[j])).x;
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float2 v = unpack2<true>(f[i]);
        x[2 * i] = v.x * scale;
        x[2 * i + 1] = v.y * scale;
      }
    }
    const int64_t to = static_cast<int64_t>(token) * a.tok[j] + head * a.head[j] + l * 16;
    if (DT == FT_DT_F32) {
      float4* dst = reinterpret_cast<float4*>(static_cast<float*>(a.out[j]) + to);
#pragma unroll
      for (int i = 0; i < 4; ++i) dst[i] = make_float4(x[4 * i], x[4 * i + 1], x[4 * i + 2], x[4 * i + 3]);
    } else {
      store32(static_cast<uint16_t*>(a.out[j]) + to, pack8<DT == FT_DT_F16>(x), pack8<DT == FT_DT_F16>(x + 8),
              a.wide_out != 0);
    }
  }
}

int ceil_log2(int n) {
  int s = 0;
  while ((1 << s) < n) ++s;
  return s;
}

bool rows_overlap_partly(const ft_rows* a, const ft_rows* b) {
  return a->base == b->base && (a->token_stride != b->token_stride || a->head_stride != b->head_stride);
}

// Shape of a write launch and the launch itself.
template <bool F16, int FMT>
ft_status launch_write(WriteArgs& a, bool interleaved, const char* what, cudaStream_t s) {
  a.half = a.rot / 2;
  const bool halves = a.half % (FMT == FT_KV_NVFP4 ? 16 : 8) == 0 && (a.D - a.rot) % 16 == 0;
  a.lanes_log2 = ceil_log2((a.D + 15) / 16);
  const int64_t items = static_cast<int64_t>(a.Hq + (FMT >= 0 ? 2 * a.Hkv : 0)) << a.lanes_log2;
  const int sms = device_sm_count();
  // Few tokens: a token's rows over several CTAs, so that each lane has one row.
  int64_t parts = (items + 127) / 128;
  if (parts > sms / a.T) parts = sms / a.T > 1 ? sms / a.T : 1;
  const int64_t per = (items + parts - 1) / parts;
  // As few rounds as leave at least 960 of the 1024 threads that fit an SM (64
  // registers): 384 lanes in one block of 384 are two blocks an SM and took 46
  // us where two rounds of 192 took 38 (8192 tokens, 32 + 2 x 8 heads of 128).
  int64_t rounds = (per + 511) / 512;
  int block = static_cast<int>(((per + rounds - 1) / rounds + 31) / 32 * 32);
  while (block > 64 && 1024 / block * block < 960) {
    ++rounds;
    block = static_cast<int>(((per + rounds - 1) / rounds + 31) / 32 * 32);
  }
  // Parts that would begin past the last row are not launched.
  a.parts = static_cast<int>(parts);
  while (a.parts > 1 && static_cast<int64_t>(a.parts - 1) * block >= items) --a.parts;
  // Many tokens: several a CTA, so that their loads overlap, and so many that
  // the CTAs fill whole waves of the SMs, as few as the batch allows (4099
  // tokens x 40 heads rotated, 456 resident CTAs: 9 a CTA 15.5 us, 8 18.7, 3
  // 16.2; 8192 tokens as above, 760 resident: 11 a CTA 35.7 us, 10 46.6, 6 36.5).
  const bool any = !(interleaved || a.rot == 0) && !halves;
  const int64_t resident = (any ? 512 : 1024) / block * sms;
  const int64_t wave_tokens = (resident > sms ? resident : sms) * kMaxBatch;
  const int64_t waves = (a.T + wave_tokens - 1) / wave_tokens;
  a.batch = static_cast<int>((a.T + waves * wave_tokens / kMaxBatch - 1) / (waves * wave_tokens / kMaxBatch));
  const int64_t groups = (a.T + a.batch - 1) / a.batch;
  FT_REQUIRE(groups * a.parts < (1ll << 31), "%s: too many rows", what);
  const unsigned grid = static_cast<unsigned>(groups) * a.parts;
  const size_t smem = static_cast<size_t>(a.batch) * 2 * ((a.half + 31) / 32 * 32) * sizeof(float);
  const auto kernel = interleaved || a.rot == 0 ? write_kernel<F16, FMT, kPairs>
                      : any                     ? write_kernel<F16, FMT, kAny>
                                                : write_kernel<F16, FMT, kHalves>;
  return launch_pdl(kernel, dim3(grid), block, smem, s, a, what);
}

template <int FMT>
ft_status launch_read(const ReadArgs& a, int32_t dtype, cudaStream_t s) {
  const uint64_t threads = static_cast<uint64_t>(a.rows) << a.lanes_log2;
  const auto kernel = dtype == FT_DT_BF16  ? read_kernel<FMT, FT_DT_BF16>
                      : dtype == FT_DT_F16 ? read_kernel<FMT, FT_DT_F16>
                                           : read_kernel<FMT, FT_DT_F32>;
  return launch_pdl(kernel, dim3(static_cast<unsigned>((threads + 255) / 256)), 256, 0, s, a, "kv_gather");
}

// Every 16 elements of 16-bit rows (D a multiple of 16) are a 32-byte place.
bool wide(const ft_rows* r) {
  return reinterpret_cast<uintptr_t>(r->base) % 32 == 0 && r->token_stride % 16 == 0 && r->head_stride % 16 == 0;
}

ft_status check_rope(const char* what, const ft_rope_table* r, int32_t D) {
  FT_REQUIRE(r->freqs != nullptr, "%s: freqs is NULL", what);
  FT_REQUIRE(r->rot_dim >= 2 && r->rot_dim % 2 == 0 && r->rot_dim <= D, "%s: rot_dim %d must be even, 2..%d", what,
             r->rot_dim, D);
  return FT_OK;
}

}  // namespace

ft_status check_rows(const char* what, const char* name, const ft_rows* r, int64_t grain) {
  FT_REQUIRE(r != nullptr && r->base != nullptr, "%s: %s is NULL", what, name);
  FT_REQUIRE(reinterpret_cast<uintptr_t>(r->base) % 16 == 0, "%s: %s not 16-byte aligned", what, name);
  FT_REQUIRE(r->token_stride % grain == 0 && r->head_stride % grain == 0 && r->token_stride >= 0 && r->head_stride >= 0,
             "%s: %s strides must be non-negative multiples of %d", what, name, static_cast<int>(grain));
  return FT_OK;
}

uint64_t kv_row_bytes(int32_t fmt, int32_t D) {
  if (D < 16 || D > 256 || D % 16) return 0;
  switch (fmt) {
    case FT_KV_BF16:
    case FT_KV_F16: return 2ull * D;
    case FT_KV_E4M3: return D;
    case FT_KV_NVFP4: return D % 32 ? 0 : D / 2;
    default: return 0;
  }
}

ft_status kv_view(const char* what, const ft_kv_cache* c, const ft_page_table* p, const int32_t* seq, int32_t T,
                  KvView* out) {
  FT_REQUIRE(c != nullptr && p != nullptr, "%s: cache or page table is NULL", what);
  const uint64_t bytes = kv_row_bytes(c->fmt, c->D);
  if (bytes == 0) return fail(FT_ERR_UNSUPPORTED, "%s: unsupported cache format %d with D = %d", what, c->fmt, c->D);
  FT_REQUIRE(c->Hkv > 0 && c->page_size > 0 && c->n_pages > 0, "%s: Hkv, page_size and n_pages must be positive", what);
  FT_REQUIRE(c->page_stride >= 0 && c->head_stride >= 0 && c->slot_stride >= 0, "%s: negative cache stride", what);
  const double last = static_cast<double>(c->n_pages - 1) * c->page_stride +
                      static_cast<double>(c->Hkv - 1) * c->head_stride +
                      static_cast<double>(c->page_size - 1) * c->slot_stride;
  if (!(last < 2147483647.0) || c->n_pages >= (1ll << 31) || c->page_stride >= (1ll << 32) ||
      c->head_stride >= (1ll << 32) || c->slot_stride >= (1ll << 32))
    return fail(FT_ERR_UNSUPPORTED, "%s: cache rows beyond 2^31", what);
  const bool quant = c->fmt == FT_KV_E4M3 || c->fmt == FT_KV_NVFP4;
  FT_REQUIRE(c->k != nullptr && c->v != nullptr, "%s: cache k or v is NULL", what);
  FT_REQUIRE(!quant || (c->k_scale != nullptr && c->v_scale != nullptr), "%s: the format needs scale arrays", what);
  FT_REQUIRE(c->fmt != FT_KV_NVFP4 || (c->k_block != nullptr && c->v_block != nullptr),
             "%s: the format needs block scale arrays", what);
  for (const void* q : {static_cast<const void*>(c->k), static_cast<const void*>(c->v),
                        static_cast<const void*>(c->k_scale), static_cast<const void*>(c->v_scale),
                        static_cast<const void*>(c->k_block), static_cast<const void*>(c->v_block)})
    FT_REQUIRE(reinterpret_cast<uintptr_t>(q) % 16 == 0, "%s: cache arrays must be 16-byte aligned", what);
  // calls of no tokens look nothing up, and may have a table of no sequences
  FT_REQUIRE(T == 0 || (p->pages != nullptr && p->max_pages > 0 && p->n_seqs > 0 && p->stride >= 0), "%s: bad page table",
             what);
  FT_REQUIRE(seq != nullptr || T <= p->n_seqs, "%s: %d rows but a page table of %d sequences", what, T, p->n_seqs);
  KvView v;
  v.data[0] = static_cast<uint8_t*>(c->k);
  v.data[1] = static_cast<uint8_t*>(c->v);
  v.scale[0] = c->k_scale;
  v.scale[1] = c->v_scale;
  v.block[0] = c->k_block;
  v.block[1] = c->v_block;
  v.at.page_size = static_cast<uint32_t>(c->page_size);
  v.at.by_page = make_fast_div(v.at.page_size);
  v.at.n_pages = static_cast<uint32_t>(c->n_pages);
  v.at.page_stride = static_cast<uint32_t>(c->page_stride);
  v.at.head_stride = static_cast<uint32_t>(c->head_stride);
  v.at.slot_stride = static_cast<uint32_t>(c->slot_stride);
  v.pages = p->pages;
  v.table_stride = p->stride;
  v.max_pages = static_cast<uint32_t>(p->max_pages);
  v.n_seqs = static_cast<uint32_t>(p->n_seqs);
  v.seq = seq;
  v.row_bytes = static_cast<int32_t>(bytes);
  v.D = c->D;
  v.Hkv = c->Hkv;
  *out = v;
  return FT_OK;
}

}  // namespace ft

using namespace ft;

extern "C" {

uint64_t ft_kv_row_bytes(int32_t fmt, int32_t D) { return kv_row_bytes(fmt, D); }

ft_status ft_rope_freqs(int32_t rot_dim, double base, int32_t scaling, double factor, double low, double high,
                        int32_t orig_len, int64_t* freqs_host) {
  FT_REQUIRE(freqs_host != nullptr, "rope_freqs: NULL pointer");
  FT_REQUIRE(rot_dim >= 2 && rot_dim % 2 == 0, "rope_freqs: rot_dim %d must be even and at least 2", rot_dim);
  FT_REQUIRE(base >= 1.0 && isfinite(base), "rope_freqs: base must be at least 1");
  FT_REQUIRE(scaling >= FT_ROPE_PLAIN && scaling <= FT_ROPE_PARTS_BY_INDEX, "rope_freqs: scaling %d", scaling);
  const bool parts = scaling == FT_ROPE_PARTS_BY_TURNS || scaling == FT_ROPE_PARTS_BY_INDEX;
  if (scaling != FT_ROPE_PLAIN)
    FT_REQUIRE(factor >= 1.0 && isfinite(factor), "rope_freqs: factor must be at least 1");
  if (parts)
    FT_REQUIRE(low > 0 && high > low && isfinite(high) && orig_len > 0,
               "rope_freqs: parts need 0 < low < high and orig_len > 0");
  FT_REQUIRE(scaling != FT_ROPE_BASE || rot_dim > 2, "rope_freqs: a base change needs rot_dim > 2");
  FT_REQUIRE(scaling != FT_ROPE_PARTS_BY_INDEX || base > 1.0, "rope_freqs: parts by index need base > 1");
  const double two_pi = 6.283185307179586476925287;
  if (scaling == FT_ROPE_BASE) base *= pow(factor, static_cast<double>(rot_dim) / (rot_dim - 2));
  // the (real) channel index whose frequency makes n turns in orig_len
  const auto index_of = [&](double n) { return rot_dim * log(orig_len / (n * two_pi)) / (2.0 * log(base)); };
  double from = 0, to = 0;
  if (scaling == FT_ROPE_PARTS_BY_INDEX) {
    from = fmax(floor(index_of(high)), 0.0);
    to = fmin(ceil(index_of(low)), rot_dim - 1.0);
    if (to <= from) to = from + 1e-3;
  }
  for (int i = 0; i < rot_dim / 2; ++i) {
    double f = pow(base, -2.0 * i / rot_dim);
    if (scaling == FT_ROPE_LINEAR) f /= factor;
    if (parts) {
      double g = scaling == FT_ROPE_PARTS_BY_TURNS ? (orig_len * f / two_pi - low) / (high - low)
                                                   : 1.0 - (i - from) / (to - from);
      g = fmin(fmax(g, 0.0), 1.0);
      f *= g + (1.0 - g) / factor;
    }
    // at most 1 radian, so below 2^62 in units of 2^-64 turn
    freqs_host[i] = static_cast<int64_t>(nearbyint(ldexp(f / two_pi, 64)));
  }
  return FT_OK;
}

ft_status ft_rope(const ft_rows* x_host, int32_t T, int32_t heads, int32_t D, int32_t dtype, const int32_t* pos,
                  const ft_rope_table* rope_host, const ft_rows* out_host, void* stream) {
  FT_REQUIRE(T >= 0 && heads >= 0, "rope: T %d, heads %d", T, heads);
  FT_REQUIRE(D >= 8 && D <= 256 && D % 8 == 0, "rope: D %d must be a multiple of 8, at most 256", D);
  FT_REQUIRE(dtype == FT_DT_BF16 || dtype == FT_DT_F16, "rope: dtype %d", dtype);
  if (T == 0 || heads == 0) return FT_OK;
  FT_REQUIRE(pos != nullptr && rope_host != nullptr, "rope: NULL pointer");
  ft_status st;
  if ((st = check_rope("rope", rope_host, D)) != FT_OK) return st;
  if ((st = check_rows("rope", "x", x_host, 8)) != FT_OK) return st;
  if ((st = check_rows("rope", "out", out_host, 8)) != FT_OK) return st;
  FT_REQUIRE(!rows_overlap_partly(x_host, out_host), "rope: in place needs the same strides");
  WriteArgs a = {};
  a.in[0] = static_cast<const uint16_t*>(x_host->base);
  a.in_tok[0] = x_host->token_stride;
  a.in_head[0] = x_host->head_stride;
  a.q_out = static_cast<uint16_t*>(out_host->base);
  a.out_tok = out_host->token_stride;
  a.out_head = out_host->head_stride;
  a.rope_pos = pos;
  a.freqs = rope_host->freqs;
  a.mscale = rope_host->mscale;
  a.rot = rope_host->rot_dim;
  a.T = T;
  a.Hq = heads;
  a.D = D;
  a.wide_in = wide(x_host) && D % 16 == 0;
  a.wide_out = wide(out_host);
  const bool pairs = rope_host->interleaved != 0;
  if (dtype == FT_DT_F16) return launch_write<true, -1>(a, pairs, "rope", as_stream(stream));
  return launch_write<false, -1>(a, pairs, "rope", as_stream(stream));
}

ft_status ft_kv_append(const ft_kv_cache* cache_host, const ft_rows* k_host, const ft_rows* v_host, int32_t T,
                       int32_t dtype, const ft_page_table* table_host, const int32_t* seq, const int32_t* pos,
                       const ft_rope_table* rope_host, const int32_t* rope_pos, const ft_rows* q_host, int32_t Hq,
                       const ft_rows* q_out_host, int32_t* dev_status, void* stream) {
  FT_REQUIRE(T >= 0, "kv_append: T %d", T);
  WriteArgs a = {};
  ft_status st;
  if ((st = kv_view("kv_append", cache_host, table_host, seq, T, &a.kv)) != FT_OK) return st;
  const int32_t fmt = cache_host->fmt;
  FT_REQUIRE(dtype == FT_DT_BF16 || dtype == FT_DT_F16, "kv_append: dtype %d", dtype);
  FT_REQUIRE(!(fmt == FT_KV_BF16 && dtype != FT_DT_BF16) && !(fmt == FT_KV_F16 && dtype != FT_DT_F16),
             "kv_append: a 16-bit cache takes rows of its own type");
  const bool with_q = q_host != nullptr || q_out_host != nullptr;
  FT_REQUIRE(!with_q || (rope_host != nullptr && Hq > 0), "kv_append: q needs a rotation and Hq > 0");
  if (T == 0) return FT_OK;
  FT_REQUIRE(pos != nullptr, "kv_append: pos is NULL");
  if ((st = check_rows("kv_append", "k", k_host, 8)) != FT_OK) return st;
  if ((st = check_rows("kv_append", "v", v_host, 8)) != FT_OK) return st;
  if (with_q) {
    if ((st = check_rows("kv_append", "q", q_host, 8)) != FT_OK) return st;
    if ((st = check_rows("kv_append", "q_out", q_out_host, 8)) != FT_OK) return st;
    FT_REQUIRE(!rows_overlap_partly(q_host, q_out_host), "kv_append: q in place needs the same strides");
    a.Hq = Hq;
    a.q_out = static_cast<uint16_t*>(q_out_host->base);
    a.out_tok = q_out_host->token_stride;
    a.out_head = q_out_host->head_stride;
  }
  const ft_rows* in[3] = {q_host, k_host, v_host};
  for (int i = with_q ? 0 : 1; i < 3; ++i) {
    a.in[i] = static_cast<const uint16_t*>(in[i]->base);
    a.in_tok[i] = in[i]->token_stride;
    a.in_head[i] = in[i]->head_stride;
  }
  a.wide_in = wide(k_host) && wide(v_host) && (!with_q || wide(q_host));
  a.wide_out = with_q && wide(q_out_host);
  bool pairs = false;
  if (rope_host != nullptr) {
    if ((st = check_rope("kv_append", rope_host, cache_host->D)) != FT_OK) return st;
    a.freqs = rope_host->freqs;
    a.mscale = rope_host->mscale;
    a.rot = rope_host->rot_dim;
    a.rope_pos = rope_pos ? rope_pos : pos;
    pairs = rope_host->interleaved != 0;
  }
  a.pos = pos;
  a.T = T;
  a.Hkv = cache_host->Hkv;
  a.D = cache_host->D;
  a.status = dev_status;
  cudaStream_t s = as_stream(stream);
  const char* what = "kv_append";
  switch (fmt) {
    case FT_KV_BF16: return launch_write<false, FT_KV_BF16>(a, pairs, what, s);
    case FT_KV_F16: return launch_write<true, FT_KV_F16>(a, pairs, what, s);
    case FT_KV_E4M3:
      return dtype == FT_DT_F16 ? launch_write<true, FT_KV_E4M3>(a, pairs, what, s)
                                : launch_write<false, FT_KV_E4M3>(a, pairs, what, s);
    default:
      return dtype == FT_DT_F16 ? launch_write<true, FT_KV_NVFP4>(a, pairs, what, s)
                                : launch_write<false, FT_KV_NVFP4>(a, pairs, what, s);
  }
}

ft_status ft_kv_gather(const ft_kv_cache* cache_host, const ft_page_table* table_host, const int32_t* seq,
                       const int32_t* pos, int32_t T, const ft_rows* k_out_host, const ft_rows* v_out_host,
                       int32_t dtype, int32_t* dev_status, void* stream) {
  FT_REQUIRE(T >= 0, "kv_gather: T %d", T);
  ReadArgs a = {};
  ft_status st;
  if ((st = kv_view("kv_gather", cache_host, table_host, seq, T, &a.kv)) != FT_OK) return st;
  FT_REQUIRE(dtype >= FT_DT_BF16 && dtype <= FT_DT_F32, "kv_gather: dtype %d", dtype);
  FT_REQUIRE(k_out_host != nullptr || v_out_host != nullptr, "kv_gather: no output");
  if (T == 0) return FT_OK;
  FT_REQUIRE(pos != nullptr, "kv_gather: pos is NULL");
  const ft_rows* out[2] = {k_out_host, v_out_host};
  a.wide_out = (!k_out_host || wide(k_out_host)) && (!v_out_host || wide(v_out_host));
  a.wide_in = reinterpret_cast<uintptr_t>(cache_host->k) % 32 == 0 && reinterpret_cast<uintptr_t>(cache_host->v) % 32 == 0;
  for (int j = 0; j < 2; ++j) {
    if (out[j] == nullptr) continue;
    if ((st = check_rows("kv_gather", j ? "v_out" : "k_out", out[j], dtype == FT_DT_F32 ? 4 : 8)) != FT_OK) return st;
    a.out[j] = out[j]->base;
    a.tok[j] = out[j]->token_stride;
    a.head[j] = out[j]->head_stride;
  }
  FT_REQUIRE(static_cast<int64_t>(T) * cache_host->Hkv < (1ll << 31), "kv_gather: too many rows");
  a.pos = pos;
  a.by_heads = make_fast_div(static_cast<uint32_t>(cache_host->Hkv));
  a.rows = static_cast<uint32_t>(T) * cache_host->Hkv;
  a.lanes_log2 = ceil_log2(cache_host->D / 16);
  a.status = dev_status;
  cudaStream_t s = as_stream(stream);
  switch (cache_host->fmt) {
    case FT_KV_BF16: return launch_read<FT_KV_BF16>(a, dtype, s);
    case FT_KV_F16: return launch_read<FT_KV_F16>(a, dtype, s);
    case FT_KV_E4M3: return launch_read<FT_KV_E4M3>(a, dtype, s);
    default: return launch_read<FT_KV_NVFP4>(a, dtype, s);
  }
}

}  // extern "C"
