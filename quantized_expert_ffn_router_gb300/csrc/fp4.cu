// fp4.cu -- rows quantised to microscaled 4-bit matrices, and read back.
//
// Both stream: each value is read once and written once (2 to 4 bytes on one
// side, 0.53 or 0.56 on the other), and HBM bounds long calls.  A thread takes
// chunks of 16 values, a whole NVFP4 block or half an MXFP4 one, so that a
// block's maximum stays in one or two lanes, loads are of 32 bytes and codes of
// 8; a row's maximum is a few shuffles, and a word a warp in shared memory where
// a row has several warps.
//
// Measured (GPU time in a graph, inputs beyond L2; of 6.79 TB/s):
//   8192 x 4096 bf16 to NVFP4 with row scales 17.6 us (72%: instructions, of which
//     65% of the issue slots are used, and the row's maximum between loads and
//     codes), f32 25.2 (90%), to MXFP4 15.2 (82%); 20480 x 2560 by a given scale
//     25.0 (79%); rows of more than 16384 values, read twice: 4096 x 20480 f32 116.8
//     (48%, each value counted once);
//   read back as bf16: 8192 x 4096 15.4 us (82%), 20480 x 2560 24.0 (83%);
//   one row of 2048: 1.2 and 1.0 us.
#include <algorithm>
#include <type_traits>

#include "ft_fp4.cuh"
#include "ft_narrow.cuh"

namespace ft {
namespace {

struct RowArgs {
  const void* x;    // quantise: the rows; values: unused
  void* out;        // values: the rows
  int64_t stride;   // elements
  uint8_t* codes;
  uint8_t* scales;
  float* scale;
  int64_t pitch, scale_stride;
  uint32_t rows;
  int32_t chunks;   // of 16 values in a row
  int32_t blocks;   // block scales of a row
  int32_t group_log2;  // values: threads of a row
  int32_t group, block_rows;  // quantise: threads of a row, rows of a block
  int32_t tiles;    // order FT_FP4_TILES
  int32_t wide;     // every 16 elements are a 32-byte place
};

// 16 values of a row, as loaded.
template <int DT>
struct Chunk {
  uint4 w[DT == FT_DT_F32 ? 4 : 2];
};

template <int DT>
__device__ __forceinline__ Chunk<DT> load_chunk(const RowArgs& a, uint32_t row, int c) {
  Chunk<DT> r;
  constexpr int kSize = DT == FT_DT_F32 ? 4 : 2;
  const uint8_t* p = static_cast<const uint8_t*>(a.x) + (static_cast<int64_t>(row) * a.stride + c * int64_t{16}) * kSize;
#pragma unroll
  for (int i = 0; i < (kSize == 4 ? 4 : 2); i += 2) load32(p + 16 * i, r.w[i], r.w[i + 1], a.wide != 0);
  return r;
}

template <int DT>
__device__ __forceinline__ void values_of(const Chunk<DT>& c, float (&x)[16]) {
  if constexpr (DT == FT_DT_F32) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[4 * i] = __uint_as_float(c.w[i].x);
      x[4 * i + 1] = __uint_as_float(c.w[i].y);
      x[4 * i + 2] = __uint_as_float(c.w[i].z);
      x[4 * i + 3] = __uint_as_float(c.w[i].w);
    }
  } else {
    unpack8<DT == FT_DT_F16>(c.w[0], x);
    unpack8<DT == FT_DT_F16>(c.w[1], x + 8);
  }
}

constexpr float kLargest = 3.4028235e38f;

// The largest magnitude of 16 values, NaN where one is NaN.
template <int DT>
__device__ __forceinline__ float chunk_max(const Chunk<DT>& c) {
  if constexpr (DT == FT_DT_F32) {  // magnitudes order as their bits do, and NaN come last
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      m = max(max(m, max(c.w[i].x & 0x7fffffffu, c.w[i].y & 0x7fffffffu)), max(c.w[i].z & 0x7fffffffu, c.w[i].w & 0x7fffffffu));
    return __uint_as_float(m);
  } else {
    using T2 = std::conditional_t<DT == FT_DT_F16, __half2, __nv_bfloat162>;
    const auto at = [&](int i) {
      const uint4& v = c.w[i >> 2];
      const uint32_t w = (i & 3) == 0 ? v.x : (i & 3) == 1 ? v.y : (i & 3) == 2 ? v.z : v.w;
      return __habs2(*reinterpret_cast<const T2*>(&w));
    };
    T2 m = __hmax2_nan(at(0), at(1));
#pragma unroll
    for (int i = 2; i < 8; ++i) m = __hmax2_nan(m, at(i));
    if constexpr (DT == FT_DT_F16) return __half2float(__hmax_nan(__low2half(m), __high2half(m)));
    else return __bfloat162float(__hmax_nan(__low2bfloat16(m), __high2bfloat16(m)));
  }
}

// The same of finite values alone.
__device__ __forceinline__ float finite_max(const float (&x)[16]) {
  float m = 0.f;
#pragma unroll
  for (int i = 0; i < 16; ++i) m = fmaxf(m, finite_abs(x[i]));
  return m;
}

__device__ __forceinline__ bool any_nan(const float (&x)[16]) {
  bool n = false;
#pragma unroll
  for (int i = 0; i < 16; ++i) n |= isnan(x[i]);
  return n;
}

// Two floats as one operand of the packed fp32 instructions.
__device__ __forceinline__ uint64_t pair(float a, float b) {
  uint64_t p;
  asm("mov.b64 %0, {%1, %2};" : "=l"(p) : "f"(a), "f"(b));
  return p;
}
__device__ __forceinline__ float2 unpair(uint64_t p) {
  float2 v;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(v.x), "=f"(v.y) : "l"(p));
  return v;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}

// Codes of 8 values.
__device__ __forceinline__ uint32_t codes8(const float* q) {
  uint32_t w;
  asm("{\n .reg .b8 c0, c1, c2, c3;\n cvt.rn.satfinite.e2m1x2.f32 c0, %2, %1;\n cvt.rn.satfinite.e2m1x2.f32 c1, %4, %3;\n"
      " cvt.rn.satfinite.e2m1x2.f32 c2, %6, %5;\n cvt.rn.satfinite.e2m1x2.f32 c3, %8, %7;\n mov.b32 %0, {c0, c1, c2, c3};\n}"
      : "=r"(w)
      : "f"(q[0]), "f"(q[1]), "f"(q[2]), "f"(q[3]), "f"(q[4]), "f"(q[5]), "f"(q[6]), "f"(q[7]));
  return w;
}
__device__ __forceinline__ uint2 codes16(const float (&q)[16]) { return make_uint2(codes8(q), codes8(q + 8)); }

// x / d for a d of at most 4 bits, as far as borders between codes of at most 4
// bits go, with an r of 1 / d (1 + 2^-22 or less): a product with the reciprocal
// and one correction step (Markstein).  y = fl(x r) is within 2^-21 of x / d; x -
// y d is exact in an fma, because d has few bits; so y + (x - y d) r is x / d
// within 2^-43 of it, and is rounded once.  A border times d has at most 8
// bits.  Where x is that product, the quotient is the border itself; else x is an
// ulp of x away at least, which is more than 0.53 ulp of the quotient, and does not
// round to the border.  So codes are those of x / d.  (With divisions,
// 8192 x 4096 bf16 took 23.1 us.)
__device__ __forceinline__ float over(float x, float r, float d) {
  const float y = x * r;
  return fmaf(fmaf(-y, d, x), r, y);
}

__device__ __forceinline__ uint2 codes_over(const float (&x)[16], float r, float d) {
  float q[16];
  const uint64_t rr = pair(r, r), dd = pair(-d, -d);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint64_t v = pair(x[2 * i], x[2 * i + 1]), y = mul2(v, rr);
    const float2 z = unpair(fma2(fma2(y, dd, v), rr, y));
    q[2 * i] = z.x;
    q[2 * i + 1] = z.y;
  }
  return codes16(q);
}

__device__ __forceinline__ float reciprocal(float x) {  // to 1 ulp
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// What a chunk becomes: its codes and its block's scale.
struct Coded {
  uint2 code;
  uint32_t byte;
};

// A chunk of NVFP4 whose largest finite magnitude is m: x is scaled by 1 / up =
// down where FOUND (powers of two), else x is scaled already.
template <bool FOUND>
__device__ __forceinline__ Coded code_nvfp4(const float (&x)[16], float m, float up, float down) {
  Coded c;
  c.byte = to_e4m3x2(over(FOUND ? m * down : m, 1.f / 6.f, 6.f), 0.f) & 0xffu;
  const float b = e4m3_value(c.byte);
  // without a block scale all codes are 0: the quotients, not their remainders, are NaN else
  const float r = b > 0.f ? reciprocal(b) : 0.f;
  c.code = codes_over(x, FOUND ? r * down : r, FOUND ? b * up : b);
  if (b == 0.f) c.code = make_uint2(0, 0);
  return c;
}

// The same of a chunk that holds infinities or NaN, not scaled yet.  (Out of
// line, and by values: as a reference, x would be in memory for every chunk.)
template <int DT, bool FOUND>
__device__ __noinline__ Coded code_odd(Chunk<DT> chunk, float up, float down) {
  Coded c;
  float x[16];
  values_of(chunk, x);
  if (!FOUND) {
#pragma unroll
    for (int i = 0; i < 16; ++i) x[i] *= down;
  }
  const float m = finite_max(x);
  if (any_nan(x)) return Coded{make_uint2(0, 0), 0x7fu};
  c.byte = to_e4m3x2(over(FOUND ? m * down : m, 1.f / 6.f, 6.f), 0.f) & 0xffu;
  const float b = e4m3_value(c.byte);
  if (b == 0.f) return Coded{make_uint2(0, 0), c.byte};
  const float r = FOUND ? reciprocal(b) * down : reciprocal(b), d = FOUND ? b * up : b;
  float q[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) q[i] = fabsf(x[i] * r) <= kLargest ? over(x[i], r, d) : x[i] * r;
  c.code = codes16(q);
  return c;
}

// FMT, DT as named; CH: chunks that a thread holds from the row's maximum to
// the codes.  0: rows longer than the block's threads hold are read twice.
// ROW: the row's scale is found (NVFP4); otherwise it is given.
//
// A block walks the rows, the next one's chunks on their way while it works on
// this one's.  Lanes past a row's last chunk, or past the last row, work on the
// last one again, and store nothing.
//
// Two chunks of fp32 and the next two are 64 registers: one block an SM (8192 x
// 12288: 76 us, 89% of HBM; 128 of two, which spill).
constexpr int blocks_of_sm(int DT, int CH) { return CH == 0 || (CH == 2 && DT == FT_DT_F32) ? 1 : 2; }
template <int FMT, int DT, int CH, bool ROW>
__global__ void __launch_bounds__(CH > 0 ? 512 : 1024, blocks_of_sm(DT, CH)) quantize_kernel(const __grid_constant__ RowArgs a) {
  __shared__ float warp_max[2][32];
  // threads of a row: a power of two of one warp's, or whole warps
  const int group = a.group, in_block = static_cast<int>(threadIdx.x) / group;
  const int l = threadIdx.x - in_block * group;
  const uint32_t step = gridDim.x * a.block_rows;
  const int last = a.chunks - 1;
  pdl_wait();
  if (a.rows <= kFewRows) pdl_launch_dependents();
  constexpr int kHeld = CH > 0 ? CH : 1;
  Chunk<DT> next[kHeld];
  const int rounds = CH > 0 ? CH : (a.chunks + group - 1) / group;
  const auto load = [&](uint32_t row, int i) {
    return load_chunk<DT>(a, min(row, a.rows - 1), min(l + i * group, last));
  };
  uint32_t base = blockIdx.x * a.block_rows;
  if (CH > 0) {
#pragma unroll
    for (int i = 0; i < kHeld; ++i) next[i] = load(base + in_block, i);
  }
  int flip = 0;
  for (; base < a.rows; base += step) {  // below 2^31 + 2^20: no overflow
    const uint32_t row = base + in_block;
    const bool live = row < a.rows;
    Chunk<DT> held[kHeld];
    if (CH > 0) {
#pragma unroll
      for (int i = 0; i < kHeld; ++i) held[i] = next[i];
#pragma unroll
      for (int i = 0; i < kHeld; ++i) next[i] = load(row + step, i);
    }
    float most[kHeld];
    float up = 1.f, down = 1.f;  // 2^e, 2^-e; given: down is fl(1 / s)
    if constexpr (ROW) {
      float m = 0.f;
#pragma unroll(CH > 0 ? CH : 1)
      for (int i = 0; i < rounds; ++i) {
        Chunk<DT> c;
        if (CH > 0) c = held[CH > 0 ? i : 0];
        else c = load(row, i);
        float mine = chunk_max(c);
        if (CH > 0) most[CH > 0 ? i : 0] = mine;
        if (!(mine <= kLargest)) {
          float x[16];
          values_of(c, x);
          mine = finite_max(x);
        }
        m = fmaxf(m, mine);
      }
      // magnitudes order as their bits do
      uint32_t bits = __float_as_uint(m);
      if (group >= 32) {
        bits = __reduce_max_sync(0xffffffffu, bits);
      } else {
        for (int o = group >> 1; o > 0; o >>= 1) bits = max(bits, __shfl_xor_sync(0xffffffffu, bits, o));
      }
      if (group > 32) {
        const int warps = group >> 5, lane = threadIdx.x & 31;
        if (lane == 0) warp_max[flip][threadIdx.x >> 5] = __uint_as_float(bits);
        __syncthreads();
        bits = __reduce_max_sync(0xffffffffu, __float_as_uint(warp_max[flip][in_block * warps + min(lane, warps - 1)]));
        flip ^= 1;
      }
      const int e = row_exponent(__uint_as_float(bits), 11, 0x280000u);  // 6 * 448 = 1.3125 * 2^11
      up = pow2f(e);
      down = pow2f(-e);
      if (live && l == 0) a.scale[row * a.scale_stride] = up;
    } else if (FMT == FT_FP4_NVFP4 && a.scale != nullptr) {
      down = __frcp_rn(a.scale[(live ? row : 0) * a.scale_stride]);
    }
    uint8_t* const codes = a.codes + row * a.pitch;
    const uint32_t r7 = row & 127;
    uint8_t* const scales = a.scales + (a.tiles ? int64_t{row >> 7} * ((a.blocks + 3) >> 2) * 512 + (r7 & 31) * 16 + (r7 >> 5) * 4
                                                : int64_t{row} * a.blocks);
    constexpr int kPer = FMT == FT_FP4_NVFP4 ? 1 : 2;  // chunks of a block
#pragma unroll(CH > 0 ? CH : 1)
    for (int i = 0; i < rounds; ++i) {
      Chunk<DT> c;
      if (CH > 0) c = held[CH > 0 ? i : 0];
      else c = load(row, i);
      const int at = l + i * group;
      float x[16];
      values_of(c, x);
      float m = ROW && CH > 0 ? most[CH > 0 ? i : 0] : chunk_max(c);
      Coded out;
      if constexpr (FMT == FT_FP4_NVFP4) {
        if (!ROW) {
          m *= fabsf(down);  // the greatest value's product is the greatest
#pragma unroll
          for (int j = 0; j < 16; ++j) x[j] *= down;
        }
        if (__any_sync(0xffffffffu, !(m <= kLargest)))
          out = code_odd<DT, ROW>(c, up, down);
        else
          out = code_nvfp4<ROW>(x, m, up, down);
      } else {
        bool nan = false;
        if (!(m <= kLargest)) {
          m = finite_max(x);
          nan = any_nan(x);
        }
        m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 1));
        nan |= __shfl_xor_sync(0xffffffffu, nan ? 1 : 0, 1) != 0;
        const int top = max(static_cast<int>(__float_as_uint(m) >> 23) - 129, -127);  // floor(log2 m) - 2
        out.byte = nan ? 0xffu : static_cast<uint32_t>(top + 127);
        const float per = __uint_as_float(static_cast<uint32_t>(127 - top) << 23);  // 2^-top: an exact product
#pragma unroll
        for (int j = 0; j < 16; ++j) x[j] *= per;
        out.code = codes16(x);
        if (nan) out.code = make_uint2(0, 0);
      }
      const bool in = live && at <= last;
      if (in) *reinterpret_cast<uint2*>(codes + at * int64_t{8}) = out.code;
      const int block = at / kPer;
      if (a.tiles) {
        // four scales a word, by one lane of four (or eight); 0 past the row's last
        uint32_t word = at <= last && at % kPer == 0 ? out.byte << (8 * (block & 3)) : 0;
        word |= __shfl_xor_sync(0xffffffffu, word, kPer);
        word |= __shfl_xor_sync(0xffffffffu, word, 2 * kPer);
        if (in && at % (4 * kPer) == 0) *reinterpret_cast<uint32_t*>(scales + (block >> 2) * int64_t{512}) = word;
      } else if (in && at % kPer == 0) {
        scales[block] = static_cast<uint8_t>(out.byte);
      }
    }
  }
}

// The values of a chunk: code * block scale is exact in fp32 (6 bits).
template <int FMT, int DT>
__global__ void __launch_bounds__(256) values_kernel(const __grid_constant__ RowArgs a) {
  const int group = 1 << a.group_log2;
  const uint32_t row = blockIdx.x * (256 >> a.group_log2) + (threadIdx.x >> a.group_log2);
  pdl_wait();
  if (a.rows <= kFewRows) pdl_launch_dependents();
  if (row >= a.rows) return;
  float s = 1.f;
  if (FMT == FT_FP4_NVFP4 && a.scale != nullptr) s = a.scale[static_cast<int64_t>(row) * a.scale_stride];
  const uint8_t* codes = a.codes + static_cast<int64_t>(row) * a.pitch;
  constexpr int kSize = DT == FT_DT_F32 ? 4 : 2;
  uint8_t* out = static_cast<uint8_t*>(a.out) + static_cast<int64_t>(row) * a.stride * kSize;
  for (int at = threadIdx.x & (group - 1); at < a.chunks; at += group) {
    const int block = FMT == FT_FP4_NVFP4 ? at : at >> 1;
    const int64_t place = a.tiles ? (static_cast<int64_t>(row >> 7) * ((a.blocks + 3) >> 2) + (block >> 2)) * 512 +
                                        (row & 31) * 16 + ((row & 127) >> 5) * 4 + (block & 3)
                                  : static_cast<int64_t>(row) * a.blocks + block;
    const uint32_t byte = a.scales[place];
    const uint2 w = *reinterpret_cast<const uint2*>(codes + static_cast<int64_t>(at) * 8);
    float b;
    if (FMT == FT_FP4_NVFP4)
      b = e4m3_value(byte);
    else  // 2^-127 has no normal fp32
      b = byte == 0 ? 0x1p-127f : __uint_as_float(byte == 0xffu ? 0x7fc00000u : byte << 23);
    uint32_t h[8];
    e2m1x8(w.x, h);
    e2m1x8(w.y, h + 4);
    float x[16];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float2 v = unpack2<true>(h[i]);
      x[2 * i] = v.x * b * s;
      x[2 * i + 1] = v.y * b * s;
    }
    uint8_t* to = out + static_cast<int64_t>(at) * 16 * kSize;
    if constexpr (DT == FT_DT_F32) {
#pragma unroll
      for (int i = 0; i < 4; i += 2) {
        const uint32_t* v = reinterpret_cast<const uint32_t*>(x + 4 * i);
        store32(to + 16 * i, make_uint4(v[0], v[1], v[2], v[3]), make_uint4(v[4], v[5], v[6], v[7]), a.wide != 0);
      }
    } else {
      store32(to, pack8<DT == FT_DT_F16>(x), pack8<DT == FT_DT_F16>(x + 8), a.wide != 0);
    }
  }
}

int ceil_log2(int64_t n) {
  int s = 0;
  while ((int64_t{1} << s) < n) ++s;
  return s;
}

template <int FMT, int DT, bool ROW>
ft_status launch_quantize(RowArgs& a, cudaStream_t s) {
  // Long calls: two chunks a thread where that leaves fewer lanes idle, or as
  // many, so that a row's maximum costs fewer steps; short ones: one, so that more
  // threads share the row.
  const int sms = device_sm_count();
  const int warps1 = (a.chunks + 31) / 32, warps2 = (a.chunks + 63) / 64;
  int ch = 1;
  if (DT != FT_DT_F32 && static_cast<int64_t>(a.rows) * a.chunks > static_cast<int64_t>(sms) * 2048 && warps2 * 2 <= warps1) ch = 2;
  if (warps1 > 16) ch = warps2 <= 16 ? 2 : 0;
  // Blocks of about 128 threads where they meet for a row's maximum, else of 512
  // (8192 x 4096: 17.4 us, of 256 18.1; 20480 x 2560 by a given scale: 26.9, 29.7).
  const int aim = ROW ? 128 : 512;
  int block;
  if (ch == 0) {
    a.group = block = 1024;
  } else if (warps1 == 1) {
    a.group = std::max(8, 1 << ceil_log2(a.chunks));  // an MXFP4 word of scales is of 8 lanes
    block = aim;
  } else {
    a.group = 32 * (ch == 2 ? warps2 : warps1);
    block = a.group * std::max(1, aim / a.group);
  }
  a.block_rows = block / a.group;
  const int64_t blocks = (static_cast<int64_t>(a.rows) + a.block_rows - 1) / a.block_rows;
  const int64_t resident = static_cast<int64_t>(sms) * std::max(1, (ch == 0 ? 1024 : 512 * blocks_of_sm(DT, ch)) / block);
  const dim3 grid(static_cast<unsigned>(std::min(blocks, resident)));
  const auto kernel = ch == 1   ? quantize_kernel<FMT, DT, 1, ROW>
                      : ch == 2 ? quantize_kernel<FMT, DT, 2, ROW>
                                : quantize_kernel<FMT, DT, 0, ROW>;
  return launch_pdl(kernel, grid, block, 0, s, a, "fp4_quantize");
}

template <int FMT, bool ROW>
ft_status quantize_typed(RowArgs& a, int32_t dtype, cudaStream_t s) {
  switch (dtype) {
    case FT_DT_BF16: return launch_quantize<FMT, FT_DT_BF16, ROW>(a, s);
    case FT_DT_F16: return launch_quantize<FMT, FT_DT_F16, ROW>(a, s);
    default: return launch_quantize<FMT, FT_DT_F32, ROW>(a, s);
  }
}

template <int FMT>
ft_status launch_values(RowArgs& a, int32_t dtype, cudaStream_t s) {
  int log2 = ceil_log2(a.chunks);
  if (log2 > 8) log2 = 8;
  a.group_log2 = log2;
  const uint32_t per_block = 256u >> log2;
  const dim3 grid((a.rows + per_block - 1) / per_block);
  const auto kernel = dtype == FT_DT_BF16  ? values_kernel<FMT, FT_DT_BF16>
                      : dtype == FT_DT_F16 ? values_kernel<FMT, FT_DT_F16>
                                           : values_kernel<FMT, FT_DT_F32>;
  return launch_pdl(kernel, grid, 256, 0, s, a, "fp4_values");
}

// The dense rows and the matrix as kernel arguments.
ft_status row_args(const char* what, const char* name, const void* dense, int64_t stride, int32_t dtype,
                   const ft_fp4_matrix* m, RowArgs* a) {
  ft_status st;
  if ((st = check_fp4(what, "matrix", m)) != FT_OK) return st;
  FT_REQUIRE(dtype >= FT_DT_BF16 && dtype <= FT_DT_F32, "%s: dtype %d", what, dtype);
  if (m->rows == 0) return FT_OK;
  const int64_t grain = dtype == FT_DT_F32 ? 4 : 8;
  FT_REQUIRE(dense != nullptr, "%s: %s is NULL", what, name);
  FT_REQUIRE(reinterpret_cast<uintptr_t>(dense) % 16 == 0, "%s: %s not 16-byte aligned", what, name);
  FT_REQUIRE(stride >= 0 && stride % grain == 0, "%s: %s stride must be a non-negative multiple of %d", what, name,
             static_cast<int>(grain));
  *a = RowArgs{};
  a->x = dense;
  a->out = const_cast<void*>(dense);
  a->stride = stride;
  a->codes = m->codes;
  a->scales = m->scales;
  a->scale = m->scale;
  a->pitch = m->pitch;
  a->scale_stride = m->scale_stride;
  a->rows = static_cast<uint32_t>(m->rows);
  a->chunks = static_cast<int32_t>(m->K / 16);
  a->blocks = static_cast<int32_t>(m->K / fp4_block(m->fmt));
  a->tiles = m->order == FT_FP4_TILES;
  a->wide = reinterpret_cast<uintptr_t>(dense) % 32 == 0 && stride % (2 * grain) == 0;
  return FT_OK;
}

}  // namespace

ft_status check_fp4(const char* what, const char* name, const ft_fp4_matrix* m) {
  FT_REQUIRE(m != nullptr, "%s: %s is NULL", what, name);
  if (m->fmt != FT_FP4_NVFP4 && m->fmt != FT_FP4_MXFP4)
    return fail(FT_ERR_UNSUPPORTED, "%s: %s: format %d", what, name, m->fmt);
  if (m->order != FT_FP4_TILES && m->order != FT_FP4_ROWS)
    return fail(FT_ERR_UNSUPPORTED, "%s: %s: order %d of the block scales", what, name, m->order);
  const int block = fp4_block(m->fmt);
  FT_REQUIRE(m->K > 0 && m->K % block == 0, "%s: %s: K %lld must be a positive multiple of %d", what, name,
             static_cast<long long>(m->K), block);
  FT_REQUIRE(m->rows >= 0, "%s: %s: rows %lld", what, name, static_cast<long long>(m->rows));
  if (m->K >= (1ll << 31) || m->rows >= (1ll << 31))
    return fail(FT_ERR_UNSUPPORTED, "%s: %s: rows or K beyond 2^31", what, name);
  if (m->rows == 0) return FT_OK;
  FT_REQUIRE(m->codes != nullptr && m->scales != nullptr, "%s: %s: codes or scales are NULL", what, name);
  FT_REQUIRE(reinterpret_cast<uintptr_t>(m->codes) % 16 == 0 && reinterpret_cast<uintptr_t>(m->scales) % 16 == 0,
             "%s: %s: codes and scales must be 16-byte aligned", what, name);
  FT_REQUIRE(m->pitch % 16 == 0 && m->pitch >= m->K / 2, "%s: %s: pitch must be whole 16 bytes and hold a row", what, name);
  FT_REQUIRE(m->fmt == FT_FP4_NVFP4 || m->scale == nullptr, "%s: %s: MXFP4 has no scale beside its blocks'", what, name);
  FT_REQUIRE(reinterpret_cast<uintptr_t>(m->scale) % 4 == 0 && m->scale_stride >= 0, "%s: %s: bad scale", what, name);
  return FT_OK;
}

}  // namespace ft

using namespace ft;

extern "C" {

uint64_t ft_fp4_scale_bytes(int32_t fmt, int32_t order, int64_t rows, int64_t K) {
  if (fmt != FT_FP4_NVFP4 && fmt != FT_FP4_MXFP4) return 0;
  const int block = fp4_block(fmt);
  if (rows <= 0 || rows >= (1ll << 31) || K <= 0 || K >= (1ll << 31) || K % block) return 0;
  const uint64_t n = static_cast<uint64_t>(K / block);
  if (order == FT_FP4_ROWS) return static_cast<uint64_t>(rows) * n;
  if (order != FT_FP4_TILES) return 0;
  return static_cast<uint64_t>((rows + kScaleTileRows - 1) / kScaleTileRows) *
         ((n + kScaleTileBlocks - 1) / kScaleTileBlocks) * 512;
}

ft_status ft_fp4_quantize(const void* x, int64_t stride, int32_t dtype, const ft_fp4_matrix* m_host, int32_t given,
                          void* stream) {
  RowArgs a;
  ft_status st;
  if ((st = row_args("fp4_quantize", "x", x, stride, dtype, m_host, &a)) != FT_OK) return st;
  const bool find = m_host->fmt == FT_FP4_NVFP4 && !given;
  FT_REQUIRE(!find || m_host->rows == 0 || (m_host->scale != nullptr && (m_host->scale_stride > 0 || m_host->rows == 1)),
             "fp4_quantize: a scale that is not given is found for each row, and needs a place of its own there");
  if (m_host->rows == 0) return FT_OK;
  cudaStream_t s = as_stream(stream);
  if (m_host->fmt == FT_FP4_MXFP4) return quantize_typed<FT_FP4_MXFP4, false>(a, dtype, s);
  return find ? quantize_typed<FT_FP4_NVFP4, true>(a, dtype, s) : quantize_typed<FT_FP4_NVFP4, false>(a, dtype, s);
}

ft_status ft_fp4_values(const ft_fp4_matrix* m_host, void* out, int64_t stride, int32_t dtype, void* stream) {
  RowArgs a;
  ft_status st;
  if ((st = row_args("fp4_values", "out", out, stride, dtype, m_host, &a)) != FT_OK) return st;
  FT_REQUIRE(m_host->rows <= 1 || stride >= m_host->K, "fp4_values: rows of out overlap");
  if (m_host->rows == 0) return FT_OK;
  return m_host->fmt == FT_FP4_NVFP4 ? launch_values<FT_FP4_NVFP4>(a, dtype, as_stream(stream))
                                     : launch_values<FT_FP4_MXFP4>(a, dtype, as_stream(stream));
}

}  // extern "C"
