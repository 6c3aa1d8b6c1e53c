// Block-wise e4m3 codes of activations: one scale for each 128 columns of a row.
//
// Quamba2, abstract: the 8-bit activations of the projections around the recurrence, here in the block-wise
// floating point code.
//     s = fl32(absmax * fl32(1/448)), 0 -> 1, within [2^-60, 2^60];    code = e4m3 value nearest to x / s
//
// Bound by the bytes. Sixteen lanes own a block, 8 columns each; a wave reads 4 neighbouring blocks of a row (1 KB of
// fp16), a workgroup 8 rows of them. The lanes' absmax is joined by lane permutations. 16384 x 4096 fp16: 40.6 us,
// 5.0 TB/s (a 1 GiB copy reaches 5.1); rows of a wave 1 / 2 / 4 / 8, among other calls: 51 / 47 / 48 / 52 us.
#include <hip/hip_runtime.h>

#include <type_traits>

#include "common.hpp"
#include "sequences.hpp"

using namespace qssm;

namespace {

struct QuantParams {
  const void* x;
  int64_t xs, cs, ss, M;
  int32_t K, wide;  // columns; units of 4 blocks in a row
  uint8_t* codes;
  float* scales;
};

constexpr int kRowsPer = 2;  // rows of a wave

template <typename T>
__device__ __forceinline__ float as_float(T v) {
  if constexpr (std::is_same_v<T, uint16_t>) return __half2float(__ushort_as_half(v));
  else return __uint_as_float(v);
}

typedef unsigned short v2u __attribute__((ext_vector_type(2)));

// x of the lane that differs in one bit of its number, as dpp_partner.
template <int STEP>
__device__ __forceinline__ uint32_t partner(uint32_t x) {
  return __float_as_uint(dpp_partner<STEP>(__uint_as_float(x)));
}

__device__ __forceinline__ uint32_t pack4(float a, float b, float c, float d) {
  const int lo = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
  return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(c, d, lo, true);
}

// The code of one value, where the fast path leaves two.
__device__ __noinline__ uint32_t exact_code(float v, float s, float f) {
  if (v != v) return 0;
  const float a = fabsf(v), t = fminf(fabsf(f), 448.0f);
  const int w = __builtin_amdgcn_cvt_pk_fp8_f32(t * (1.0f - 0x1p-22f), fminf(t * (1.0f + 0x1p-22f), 448.0f), 0, false);
  const uint32_t lo = w & 0xFF, hi = (w >> 8) & 0xFF;
  uint32_t c = lo;
  if (lo != hi) {
    // the midpoint has 5 bits, so one rounding keeps the sign of the exact a - mid s, and its zero
    const float mid = 0.5f * (__builtin_amdgcn_cvt_f32_fp8((int)lo, 0) + __builtin_amdgcn_cvt_f32_fp8((int)hi, 0));
    const float e = fmaf(-mid, s, a);
    c = e > 0.0f ? hi : e < 0.0f ? lo : (lo & 1) ? hi : lo;
  }
  return c | (__float_as_uint(v) >> 31 << 7);
}

// VEC: whole 16-byte loads and 8-byte stores at any address; else a value at a time.
template <typename T, bool VEC>
__global__ __launch_bounds__(256) void k_quant_f8(QuantParams p) {
  const int wave = uniform(threadIdx.x >> 6), lane = threadIdx.x & 63;
  const int unit = blockIdx.x % p.wide;
  const int64_t m0 = (int64_t)(blockIdx.x / p.wide) * (4 * kRowsPer) + wave * kRowsPer;
  const int col = unit * 512 + lane * 8, block = col / 128;
  const T* x = reinterpret_cast<const T*>(p.x) + col;
  T raw[kRowsPer][8];
#pragma unroll
  for (int r = 0; r < kRowsPer; ++r) {
#pragma unroll
    for (int i = 0; i < 8; ++i) raw[r][i] = 0;
    if (m0 + r < p.M) {
      const T* at = x + (m0 + r) * p.xs;
      if (VEC) {
        if (col < p.K) __builtin_memcpy(raw[r], at, sizeof(raw[r]));
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (col + i < p.K) raw[r][i] = at[i];
      }
    }
  }
#pragma unroll
  for (int r = 0; r < kRowsPer; ++r) {
    const int64_t m = m0 + r;
    if (m >= p.M) return;
    // the largest |x| by its bits: a NaN or an infinity is larger than every number
    uint32_t most = 0;
    if constexpr (std::is_same_v<T, uint16_t>) {
      v2u pair = {0, 0};
#pragma unroll
      for (int i = 0; i < 8; i += 2) pair = __builtin_elementwise_max(pair, (v2u)(v2u{raw[r][i], raw[r][i + 1]} & v2u{0x7fff, 0x7fff}));
      most = max(pair[0], pair[1]);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) most = max(most, raw[r][i] & 0x7fffffffu);
    }
    most = max(most, partner<1>(most));
    most = max(most, partner<2>(most));
    most = max(most, partner<4>(most));
    most = max(most, partner<8>(most));
    const bool special = most >= (std::is_same_v<T, uint16_t> ? 0x7c00u : 0x7f800000u);  // one of the block is no number
    float v[8], a = as_float((T)most);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = as_float(raw[r][i]);
    if (special) {
      a = 0.0f;
#pragma unroll
      for (int i = 0; i < 8; ++i) a = fmaxf(a, finite_abs(v[i]));
      a = fmaxf(a, dpp_partner<1>(a));
      a = fmaxf(a, dpp_partner<2>(a));
      a = fmaxf(a, dpp_partner<4>(a));
      a = fmaxf(a, dpp_partner<8>(a));
    }
    const float s = a == 0.0f ? 1.0f : fminf(fmaxf(a * (1.0f / 448.0f), 0x1p-60f), 0x1p60f);
    if (col >= p.K) continue;
    if ((lane & 15) == 0) p.scales[block * p.ss + m] = s;
    // v lo and v hi lie around the quotient (lo and hi are within 2^-23 of 1 / s (1 -+ 2^-21), the products round by 2^-24): where
    // their codes are one, it is the quotient's. Both stay below 464, where e4m3 has no more number.
    const float rc = 1.0f / s, lo = rc * (1.0f - 0x1p-21f), hi = rc * (1.0f + 0x1p-21f);
    uint32_t w[2] = {pack4(v[0] * lo, v[1] * lo, v[2] * lo, v[3] * lo), pack4(v[4] * lo, v[5] * lo, v[6] * lo, v[7] * lo)};
    const bool two = w[0] != pack4(v[0] * hi, v[1] * hi, v[2] * hi, v[3] * hi) || w[1] != pack4(v[4] * hi, v[5] * hi, v[6] * hi, v[7] * hi);
    // (the largest scale: what is far beyond 448 of it goes there too)
    if (two || special || a > 450.0f * s) {
      w[0] = w[1] = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) w[i / 4] |= exact_code(v[i], s, v[i] * rc) << (8 * (i % 4));
    }
    uint8_t* out = p.codes + m * p.cs + col;
    if (VEC) {
      __builtin_memcpy(out, w, 8);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (col + i < p.K) out[i] = (uint8_t)(w[i / 4] >> (8 * (i % 4)));
    }
  }
}

constexpr int64_t kMaxBlocks = ((int64_t)1 << 24) - 1;  // a grid holds fewer than 2^32 threads

}  // namespace

extern "C" qssm_status qssm_quant_f8(const void* x, int32_t x_dtype, int64_t rows, int64_t K, int64_t x_stride,
                                     uint8_t* codes, int64_t codes_stride, float* scales, int64_t scales_stride,
                                     hipStream_t stream) {
  clear_error();
  if (rows < 0 || K < 0) return fail(QSSM_ERR_INVALID_ARG, "negative extent");
  if (x_dtype != QSSM_F32 && x_dtype != QSSM_F16) return fail(QSSM_ERR_INVALID_ARG, "x_dtype must be QSSM_F32 or QSSM_F16");
  if (rows > 0x7fffffff || K > (1 << 24)) return fail(QSSM_ERR_UNSUPPORTED, "rows above 2^31 - 1 or K above 2^24");
  const int64_t sx = type_size(x_dtype), blocks128 = cdiv(K, 128);
  if (const qssm_status s = check_rows("x", x, rows, K, x_stride, sx)) return s;
  if (const qssm_status s = check_rows("codes", codes, rows, K, codes_stride, 1)) return s;
  if (const qssm_status s = check_rows("scales", scales, blocks128, rows, scales_stride, 4)) return s;
  if (rows == 0 || K == 0) return QSSM_OK;
  if (!x || !codes || !scales) return fail(QSSM_ERR_INVALID_ARG, "null required pointer");
  const Span sp_x{x, rows, x_stride * sx, K * sx}, sp_c{codes, rows, codes_stride, K};
  const Span sp_s{scales, blocks128, scales_stride * 4, rows * 4};
  if (overlap(sp_x, sp_c) || overlap(sp_x, sp_s) || overlap(sp_c, sp_s))
    return fail(QSSM_ERR_INVALID_ARG, "x, codes and scales overlap");
  QuantParams p{x, x_stride, codes_stride, scales_stride, rows, (int32_t)K, (int32_t)cdiv(K, 512), codes, scales};
  const int64_t blocks = cdiv(rows, 4 * kRowsPer) * p.wide;
  if (blocks > kMaxBlocks) return fail(QSSM_ERR_UNSUPPORTED, "rows * K too large");
  const bool vec = K % 8 == 0;
  if (x_dtype == QSSM_F16)
    vec ? k_quant_f8<uint16_t, true><<<(unsigned)blocks, 256, 0, stream>>>(p) : k_quant_f8<uint16_t, false><<<(unsigned)blocks, 256, 0, stream>>>(p);
  else
    vec ? k_quant_f8<uint32_t, true><<<(unsigned)blocks, 256, 0, stream>>>(p) : k_quant_f8<uint32_t, false><<<(unsigned)blocks, 256, 0, stream>>>(p);
  return launch_status("quant_f8");
}
