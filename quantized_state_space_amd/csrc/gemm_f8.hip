// Linear layer in e4m3 with one scale for each row and 128 columns of the activations, and each 128 x 128 block of the
// weights, on MFMA with fp32 accumulation.
//
// Quamba2, abstract: the 8-bit projections around the recurrence, here in the block-wise floating point code.
//     y[m, n] = bias[n] + sum_b sa[b, m] sw[n / 128, b] (sum_k in b of a[m, k] w[n, k])
// Both operands have k contiguous. A lane holds row (or column) l % 32 and 32 of each 64 k; which k these are does not
// matter, since both operands are loaded alike. The weights go in as the first operand, so a lane ends with
// one token and groups of 4 consecutive output channels: the scales of a block are then one number per
// lane, and applying them one fused multiply-add per output and block.
//
// Two products: v_mfma_f32_32x32x64_f8f6f4 adds 8 neighbouring products at a time and cuts each at 2^-13 of the power of
// two of the largest (seen from 448^2 beside smaller ones; v_mfma_f32_32x32x16_fp8_fp8 gives the same bits):
// 1.4e-5 of the result for normal data, 5e-5 for codes of every exponent, a tenth of an fp16 y's own
// rounding. An fp32 y is worth more: there the codes are converted to fp16, exactly, for
// v_mfma_f32_32x32x16_f16, at half the rate, whose sums are off by 1e-8 to 6e-7.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <type_traits>

#include "common.hpp"
#include "sequences.hpp"

using namespace qssm;

namespace {

typedef int v4i __attribute__((ext_vector_type(4)));
typedef int v8i __attribute__((ext_vector_type(8)));
typedef _Float16 v2h __attribute__((ext_vector_type(2)));
typedef _Float16 v8h __attribute__((ext_vector_type(8)));
typedef float v16f __attribute__((ext_vector_type(16)));

struct GemmParams {
  int64_t M, N, K;
  const uint8_t* a;
  int64_t as;
  const float* sa;
  int64_t sas;
  const uint8_t* w;
  int64_t ws;
  const float* sw;
  const float* bias;
  void* y;
  int64_t ys;
  int32_t yf16, kb;  // blocks of K
};

// A scale in [2^-60, 2^60], 0 for another: the product of two is a normal number, and with a sum of 128 products (up
// to 2^25) it overflows only where the result does.
__device__ __forceinline__ float valid_or_zero(float s) { return s >= 0x1p-60f && s <= 0x1p60f ? s : 0.0f; }

// 16 codes of a row from k on, at any address; codes at or past K are 0 and not read.
__device__ __forceinline__ uint4 load16(const uint8_t* row, int64_t k, int64_t K) {
  uint32_t w[4] = {0u, 0u, 0u, 0u};
  if (k + 16 <= K) {
    __builtin_memcpy(w, row + k, 16);
  } else {
#pragma unroll
    for (int i = 0; i < 16; ++i)
      if (k + i < K) w[i / 4] |= (uint32_t)row[k + i] << (8 * (i % 4));
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// LDS rows of 128 bytes; the 16-byte chunk c of row r is in slot c ^ swizzle(r), which spreads the rows that a 16-byte
// read serves together over all 64 banks.
__device__ __forceinline__ int swizzle(int row) { return (row >> 1) & 7; }

__device__ __forceinline__ void put(const GemmParams& p, int64_t m, int64_t n, float v) {
  if (p.yf16) reinterpret_cast<__half*>(p.y)[m * p.ys + n] = __float2half_rn(v);
  else reinterpret_cast<float*>(p.y)[m * p.ys + n] = v;
}

// The 32 codes of a lane: row `row`, half kh of slice ks (64 codes) of a step.
__device__ __forceinline__ v8i fragment(const uint8_t* stage, int row, int ks, int kh) {
  const int c = 4 * ks + 2 * kh, x = swizzle(row);
  const v4i lo = *reinterpret_cast<const v4i*>(stage + row * 128 + ((c ^ x) * 16));
  const v4i hi = *reinterpret_cast<const v4i*>(stage + row * 128 + (((c + 1) ^ x) * 16));
  return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
}

// Eight codes as fp16, exactly (NaN codes too).
__device__ __forceinline__ v8h to_half(int lo, int hi) {
  const v2h r[4] = {__builtin_amdgcn_cvt_scalef32_pk_f16_fp8(lo, 1.0f, false), __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(lo, 1.0f, true),
                    __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(hi, 1.0f, false), __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(hi, 1.0f, true)};
  return __builtin_bit_cast(v8h, r);
}

// c + the products of a slice of 64 codes. EXACT: through fp16.
template <bool EXACT>
__device__ __forceinline__ v16f product(const v8i& w, const v8i& a, v16f c) {
  if constexpr (EXACT) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      c = __builtin_amdgcn_mfma_f32_32x32x16_f16(to_half(w[2 * i], w[2 * i + 1]), to_half(a[2 * i], a[2 * i + 1]), c, 0, 0, 0);
    return c;
  } else {
    return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(w, a, c, 0, 0, 0, 0, 0, 0);
  }
}

// Tiles of 64 x 64, a quarter a wave, with the operands through registers: rows at any address, any K.
template <bool EXACT>
__global__ __launch_bounds__(256) void k_gemm_f8_any(GemmParams p) {
  __shared__ __align__(16) uint8_t sm[2][2][64 * 128];
  const int tid = threadIdx.x, lane = tid & 63, wave = uniform(tid >> 6), kh = lane >> 5;
  const int64_t nm = (p.M + 63) / 64;
  const int64_t m0 = blockIdx.x % nm * 64, n0 = blockIdx.x / nm * 64;
  const int wm = wave & 1, wn = wave >> 1;
  const int64_t m = m0 + wm * 32 + (lane & 31), mc = min(m, p.M - 1);
  const float* sw = p.sw + n0 / 128 * p.kb;
  uint4 va[2], vw[2];
  const auto load = [&](int b) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int row = (tid + 256 * i) / 8, c = tid % 8;
      va[i] = load16(p.a + min(m0 + row, p.M - 1) * p.as, (int64_t)b * 128 + c * 16, p.K);
      vw[i] = load16(p.w + min(n0 + row, p.N - 1) * p.ws, (int64_t)b * 128 + c * 16, p.K);
    }
  };
  const auto store = [&](int st) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int row = (tid + 256 * i) / 8, c = (tid % 8) ^ swizzle(row);
      *reinterpret_cast<uint4*>(&sm[st][0][row * 128 + c * 16]) = va[i];
      *reinterpret_cast<uint4*>(&sm[st][1][row * 128 + c * 16]) = vw[i];
    }
  };
  v16f acc = v16f{};
  if (p.kb > 0) {
    load(0);
    store(0);
  }
  for (int b = 0; b < p.kb; ++b) {
    __syncthreads();
    if (b + 1 < p.kb) load(b + 1);
    const float s = valid_or_zero(p.sa[b * p.sas + mc]) * valid_or_zero(sw[b]);
    v16f part = v16f{};
#pragma unroll
    for (int ks = 0; ks < 2; ++ks)
      part = product<EXACT>(fragment(sm[b & 1][1], wn * 32 + (lane & 31), ks, kh), fragment(sm[b & 1][0], wm * 32 + (lane & 31), ks, kh), part);
#pragma unroll
    for (int i = 0; i < 16; ++i) acc[i] = fmaf(part[i], s, acc[i]);
    if (b + 1 < p.kb) store((b + 1) & 1);
  }
  if (m >= p.M) return;
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const int64_t n = n0 + wn * 32 + 8 * (i / 4) + 4 * kh + i % 4;
    if (n < p.N) put(p, m, n, acc[i] + (p.bias ? p.bias[n] : 0.0f));
  }
}

}  // namespace

extern "C" qssm_status qssm_gemm_f8(const qssm_gemm_f8_args* a, hipStream_t stream) {
  clear_error();
  if (!a) return fail(QSSM_ERR_INVALID_ARG, "args is null");
  const int64_t M = a->M, N = a->N, K = a->K;
  if (M < 0 || N < 0 || K < 0) return fail(QSSM_ERR_INVALID_ARG, "negative extent");
  if (a->y_dtype != QSSM_F32 && a->y_dtype != QSSM_F16) return fail(QSSM_ERR_INVALID_ARG, "y_dtype must be QSSM_F32 or QSSM_F16");
  if (a->reserved != 0) return fail(QSSM_ERR_INVALID_ARG, "reserved must be 0");
  if (K > (1 << 20) || M > (1 << 27) || N > (1 << 27)) return fail(QSSM_ERR_UNSUPPORTED, "K above 2^20, or M or N above 2^27");
  const int64_t kb = cdiv(K, 128), sy = type_size(a->y_dtype);
  if (const qssm_status s = check_rows("a", a->a, M, K, a->a_stride, 1)) return s;
  if (const qssm_status s = check_rows("w", a->w, N, K, a->w_stride, 1)) return s;
  if (const qssm_status s = check_rows("a_scales", a->a_scales, kb, M, a->a_scales_stride, 4)) return s;
  if (const qssm_status s = check_rows("y", a->y, M, N, a->y_stride, sy)) return s;
  if (std::max(a->a_stride, a->w_stride) > (1 << 22)) return fail(QSSM_ERR_UNSUPPORTED, "a_stride or w_stride above 2^22");
  if (M == 0 || N == 0) return QSSM_OK;
  if (!a->y || (K > 0 && (!a->a || !a->w || !a->a_scales || !a->w_scales))) return fail(QSSM_ERR_INVALID_ARG, "null required pointer");
  if (((uintptr_t)a->w_scales | (uintptr_t)a->bias) % 4 != 0)
    return fail(QSSM_ERR_INVALID_ARG, "w_scales or bias is not aligned to its type");
  // a grid holds fewer than 2^32 threads
  if (cdiv(M, 64) * cdiv(N, 64) >= (1 << 24)) return fail(QSSM_ERR_UNSUPPORTED, "M * N too large");
  const Span y{a->y, M, a->y_stride * sy, N * sy};
  if (overlap(y, Span{a->a, M, a->a_stride, K}) || overlap(y, Span{a->w, N, a->w_stride, K}) || overlap(y, flat(a->bias, N * 4)) ||
      overlap(y, Span{a->a_scales, kb, a->a_scales_stride * 4, M * 4}) || overlap(y, flat(a->w_scales, cdiv(N, 128) * kb * 4)))
    return fail(QSSM_ERR_INVALID_ARG, "y overlaps an input");
  const GemmParams p{M, N, K, a->a, a->a_stride, a->a_scales, a->a_scales_stride, a->w, a->w_stride, a->w_scales, a->bias, a->y,
                     a->y_stride, a->y_dtype == QSSM_F16, (int32_t)kb};
  const unsigned grid = (unsigned)(cdiv(M, 64) * cdiv(N, 64));
  p.yf16 ? k_gemm_f8_any<false><<<grid, 256, 0, stream>>>(p) : k_gemm_f8_any<true><<<grid, 256, 0, stream>>>(p);
  return launch_status("gemm_f8");
}
