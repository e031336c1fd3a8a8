// fp4.cu -- rows quantised to microscaled 4-bit matrices, and read back.
//
// Both stream: each value is read once and written once (2 to 4 bytes on one
// side, 0.53 or 0.56 on the other), and HBM bounds long calls.  A thread takes
// chunks of 16 values, a whole NVFP4 block or half an MXFP4 one, so that a
// block's maximum stays in one or two lanes, loads are of 32 bytes and codes of
// 8; a row's maximum is a few shuffles, and a word a warp in shared memory where
// a row has several warps.
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
  int32_t group_log2;  // threads of a row
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

// The largest magnitude of 16 values, NaN where one is NaN.  Magnitudes of the
// same type order as their bits do, and NaN come last.
template <int DT>
__device__ __forceinline__ float chunk_max(const Chunk<DT>& c) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < (DT == FT_DT_F32 ? 4 : 2); ++i) {
    const uint32_t w[4] = {c.w[i].x, c.w[i].y, c.w[i].z, c.w[i].w};
#pragma unroll
    for (int j = 0; j < 4; ++j) m = DT == FT_DT_F32 ? max(m, w[j] & 0x7fffffffu) : __vmaxu2(m, w[j] & 0x7fff7fffu);
  }
  if constexpr (DT == FT_DT_F32) return __uint_as_float(m);
  const uint32_t top = max(m >> 16, m & 0xffffu);
  return DT == FT_DT_F16 ? __half2float(__ushort_as_half(static_cast<uint16_t>(top))) : __uint_as_float(top << 16);
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

// Codes of 16 values.
__device__ __forceinline__ uint2 codes16(const float (&q)[16]) {
  uint32_t w[2] = {0, 0};
#pragma unroll
  for (int i = 0; i < 8; ++i) w[i >> 2] |= to_e2m1x2(q[2 * i], q[2 * i + 1]) << (8 * (i & 3));
  return make_uint2(w[0], w[1]);
}

// Codes of x / d for a d of few bits, with r = fl(1 / d): a product with the
// reciprocal and one correction step (Markstein).  q = fl(x r) is within 2 ulp;
// x - q d is exact in an fma, because d has 4 bits; so the corrected quotient is
// that of x / d + 2^-46 of it, rounded.  A border between two codes has at most
// 4 bits, its product with d at most 8: x is that product, and the quotient
// comes out as the border, or differs by an ulp of x at least, which is more than
// 0.53 ulp of the quotient.  Either way the code is that of x / d.
__device__ __forceinline__ uint2 codes_over(const float (&x)[16], float r, float d, bool odd) {
  float q[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const float y = x[i] * r;
    q[i] = fmaf(fmaf(-y, d, x[i]), r, y);
  }
  if (odd) {  // infinities have no remainder
#pragma unroll
    for (int i = 0; i < 16; ++i)
      if (!(fabsf(x[i] * r) <= kLargest)) q[i] = x[i] * r;
  }
  return codes16(q);
}

// FMT, DT as named; CH: chunks that a thread holds from the row's maximum to
// the codes.  0: rows longer than the block's threads hold are read twice.
// ROW: the row's scale is found (NVFP4); otherwise it is given.
template <int FMT, int DT, int CH, bool ROW>
__global__ void __launch_bounds__(1024) quantize_kernel(const __grid_constant__ RowArgs a) {
  __shared__ float warp_max[32];
  const int group = 1 << a.group_log2;
  const int l = threadIdx.x & (group - 1);
  // the launch has up to 2^31 rows of up to 2^10 threads
  const uint32_t row = blockIdx.x * (blockDim.x >> a.group_log2) + (threadIdx.x >> a.group_log2);
  const bool live = row < a.rows;
  const uint32_t r = live ? row : a.rows - 1;
  pdl_wait();
  constexpr int kHeld = CH > 0 ? CH : 1;
  Chunk<DT> held[kHeld];
  const int rounds = CH > 0 ? CH : (a.chunks + group - 1) >> a.group_log2;
  const auto load = [&](int i, Chunk<DT>& c) {
    const int at = l + (i << a.group_log2);
    if (at < a.chunks) {
      c = load_chunk<DT>(a, r, at);
    } else {
#pragma unroll
      for (auto& w : c.w) w = make_uint4(0, 0, 0, 0);
    }
  };
  if (CH > 0) {
#pragma unroll
    for (int i = 0; i < kHeld; ++i) load(i, held[i]);
  }
  int e = 0;
  float inv = 1.f;
  if constexpr (ROW) {
    float m = 0.f;
#pragma unroll(CH > 0 ? CH : 1)
    for (int i = 0; i < rounds; ++i) {
      Chunk<DT> c;
      if (CH > 0) c = held[CH > 0 ? i : 0];
      else load(i, c);
      float mine = chunk_max(c);
      if (!(mine <= kLargest)) {
        float x[16];
        values_of(c, x);
        mine = finite_max(x);
      }
      m = fmaxf(m, mine);
    }
    for (int o = min(group, 32) >> 1; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    if (group > 32) {
      const int warp = threadIdx.x >> 5, warps = group >> 5;
      if ((threadIdx.x & 31) == 0) warp_max[warp] = m;
      __syncthreads();
      m = warp_max[(warp & ~(warps - 1)) | (threadIdx.x & (warps - 1))];
      for (int o = warps >> 1; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    }
    e = row_exponent(m, 11, 0x280000u);  // 6 * 448 = 1.3125 * 2^11
    if (live && l == 0) a.scale[static_cast<int64_t>(row) * a.scale_stride] = pow2f(e);
  } else if (FMT == FT_FP4_NVFP4 && a.scale != nullptr) {
    inv = __frcp_rn(a.scale[static_cast<int64_t>(r) * a.scale_stride]);
  }
  uint8_t* const codes = a.codes + static_cast<int64_t>(r) * a.pitch;
  constexpr int kPer = FMT == FT_FP4_NVFP4 ? 1 : 2;  // chunks of a block
#pragma unroll(CH > 0 ? CH : 1)
  for (int i = 0; i < rounds; ++i) {
    Chunk<DT> c;
    if (CH > 0) c = held[CH > 0 ? i : 0];
    else load(i, c);
    const int at = l + (i << a.group_log2);
    float x[16];
    values_of(c, x);
    float m;
    if (FMT == FT_FP4_NVFP4 && !ROW) {
      m = 0.f;
#pragma unroll
      for (int j = 0; j < 16; ++j) {
        x[j] *= inv;
        m = fmaxf(m, fabsf(x[j]));
        if (isnan(x[j])) m = INFINITY;  // sorted out below
      }
    } else {
      m = chunk_max(c);
    }
    bool odd = !(m <= kLargest), nan = false;
    if (odd) {
      m = finite_max(x);
      nan = any_nan(x);
    }
    uint32_t byte;
    uint2 code;
    if constexpr (FMT == FT_FP4_NVFP4) {
      byte = to_e4m3x2(nan ? NAN : __fdiv_rn(m * pow2f(-e), 6.f), 0.f) & 0xffu;
      const float b = e4m3_value(byte);
      code = make_uint2(0, 0);
      if (b > 0.f) code = codes_over(x, __frcp_rn(b) * pow2f(-e), b * pow2f(e), odd);
    } else {
      m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 1));
      nan |= __shfl_xor_sync(0xffffffffu, nan ? 1 : 0, 1) != 0;
      const int top = max(static_cast<int>(__float_as_uint(m) >> 23) - 129, -127);  // floor(log2 m) - 2
      byte = nan ? 0xffu : static_cast<uint32_t>(top + 127);
      const float per = __uint_as_float(static_cast<uint32_t>(127 - top) << 23);  // 2^-top: an exact product
#pragma unroll
      for (int j = 0; j < 16; ++j) x[j] *= per;
      code = codes16(x);
      if (nan) code = make_uint2(0, 0);
    }
    const bool in = live && at < a.chunks;
    if (in) *reinterpret_cast<uint2*>(codes + static_cast<int64_t>(at) * 8) = code;
    const int block = at / kPer;
    if (a.tiles) {
      // four scales a word, by one lane of four (or eight); 0 past the row's last
      uint32_t word = in && at % kPer == 0 ? byte << (8 * (block & 3)) : 0;
      word |= __shfl_xor_sync(0xffffffffu, word, kPer);
      word |= __shfl_xor_sync(0xffffffffu, word, 2 * kPer);
      if (in && at % (4 * kPer) == 0) {
        const int64_t tile = static_cast<int64_t>(row >> 7) * ((a.blocks + 3) >> 2) + (block >> 2);
        *reinterpret_cast<uint32_t*>(a.scales + tile * 512 + (row & 31) * 16 + ((row & 127) >> 5) * 4) = word;
      }
    } else if (in && at % kPer == 0) {
      a.scales[static_cast<int64_t>(row) * a.blocks + block] = static_cast<uint8_t>(byte);
    }
  }
}

// The values of a chunk: code * block scale is exact in fp32 (6 bits).
template <int FMT, int DT>
__global__ void __launch_bounds__(256) values_kernel(const __grid_constant__ RowArgs a) {
  const int group = 1 << a.group_log2;
  const uint32_t row = blockIdx.x * (256 >> a.group_log2) + (threadIdx.x >> a.group_log2);
  pdl_wait();
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
  // Long calls: two chunks a thread, so that loads overlap and a row's maximum
  // costs fewer steps.  Short ones: one, so that more threads share the row.
  const int64_t work = static_cast<int64_t>(a.rows) * a.chunks;
  const int per = work > static_cast<int64_t>(device_sm_count()) * 2048 ? 2 : 1;
  int log2 = ceil_log2((a.chunks + per - 1) / per);
  if (log2 < 3) log2 = 3;  // an MXFP4 word of scales is of 8 lanes
  int ch = per;
  if (log2 > 10) {
    ch = (a.chunks + 1023) / 1024;
    log2 = 10;
  }
  a.group_log2 = log2;
  const int block = log2 > 8 ? 1 << log2 : 256;
  const uint32_t per_block = static_cast<uint32_t>(block) >> log2;
  const dim3 grid((a.rows + per_block - 1) / per_block);
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
  if (m_host->rows == 0) return FT_OK;
  return m_host->fmt == FT_FP4_NVFP4 ? launch_values<FT_FP4_NVFP4>(a, dtype, as_stream(stream))
                                     : launch_values<FT_FP4_MXFP4>(a, dtype, as_stream(stream));
}

}  // extern "C"
