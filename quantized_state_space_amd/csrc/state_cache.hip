// int8 recurrent state: rows of N values written as int8 codes with one scale each, and read back.
//
//     s = absmax(finite |h|) fl32(1/127),  q = quant8(h, s)          h' = fl32(s q)
//
// Both are passes bound by the bytes (fp32: 5 B per value each way).
#include <hip/hip_runtime.h>

#include "common.hpp"

using namespace qssm;

namespace {

constexpr int kThreads = 256;

template <bool F16>
__device__ __forceinline__ float load1(const void* h, int64_t i) {
  if constexpr (F16) return __half2float(reinterpret_cast<const __half*>(h)[i]);
  else return reinterpret_cast<const float*>(h)[i];
}

// One wave per row.
template <bool F16>
__global__ __launch_bounds__(kThreads) void k_state_quant(const void* h, int64_t rows, int64_t N,
                                                          int8_t* codes, float* scales) {
  const int lane = threadIdx.x & 63;
  const int64_t nwaves = (int64_t)gridDim.x * (kThreads / 64);
  for (int64_t row = (int64_t)blockIdx.x * (kThreads / 64) + (threadIdx.x >> 6); row < rows;
       row += nwaves) {
    float a = 0.0f;
    for (int64_t n = lane; n < N; n += 64) a = fmaxf(a, finite_abs(load1<F16>(h, row * N + n)));
#pragma unroll
    for (int off = 32; off > 0; off >>= 1) a = fmaxf(a, __shfl_xor(a, off, 64));
    const float s = row_scale(a), r = recip_or_zero(s);
    for (int64_t n = lane; n < N; n += 64) codes[row * N + n] = quant8_r(load1<F16>(h, row * N + n), s, r);
    if (lane == 0) scales[row] = s;
  }
}

template <bool F16>
__global__ __launch_bounds__(kThreads) void k_state_dequant(const int8_t* codes, const float* scales,
                                                            int64_t rows, int64_t N, void* out) {
  const int lane = threadIdx.x & 63;
  const int64_t nwaves = (int64_t)gridDim.x * (kThreads / 64);
  for (int64_t row = (int64_t)blockIdx.x * (kThreads / 64) + (threadIdx.x >> 6); row < rows;
       row += nwaves) {
    const float s = scale_ok(scales[row]) ? scales[row] : 0.0f;
    for (int64_t n = lane; n < N; n += 64) {
      float v = (float)codes[row * N + n] * s;
      // keeps the product's rounding to fp32 apart from the one to fp16 (the compiler would join
      // them in a mixed-precision fma, which rounds once)
      if constexpr (F16) asm("" : "+v"(v));
      if constexpr (F16) reinterpret_cast<__half*>(out)[row * N + n] = __float2half_rn(v);
      else reinterpret_cast<float*>(out)[row * N + n] = v;
    }
  }
}

qssm_status check(int32_t dtype, int64_t rows, int64_t N) {
  if (dtype != QSSM_F32 && dtype != QSSM_F16)
    return fail(QSSM_ERR_INVALID_ARG, "the values must be QSSM_F32 or QSSM_F16");
  if (rows < 0 || N < 1) return fail(QSSM_ERR_INVALID_ARG, "rows must be >= 0 and N >= 1");
  if (N > 0x7fffffff || rows > ((int64_t)1 << 60) / N)
    return fail(QSSM_ERR_UNSUPPORTED, "rows * N too large");
  return QSSM_OK;
}

unsigned grid_for(int64_t rows) {
  const int64_t b = cdiv(rows, kThreads / 64);
  return (unsigned)(b < 65536 ? b : 65536);
}

}  // namespace

extern "C" qssm_status qssm_state_quant(const void* h, int32_t h_dtype, int64_t rows, int64_t N,
                                        int8_t* codes, float* scales, hipStream_t stream) {
  clear_error();
  if (qssm_status st = check(h_dtype, rows, N)) return st;
  if (rows == 0) return QSSM_OK;
  if (!h || !codes || !scales) return fail(QSSM_ERR_INVALID_ARG, "null required pointer");
  if (h_dtype == QSSM_F16) k_state_quant<true><<<grid_for(rows), kThreads, 0, stream>>>(h, rows, N, codes, scales);
  else k_state_quant<false><<<grid_for(rows), kThreads, 0, stream>>>(h, rows, N, codes, scales);
  return launch_status("state_quant");
}

extern "C" qssm_status qssm_state_dequant(const int8_t* codes, const float* scales, int64_t rows,
                                          int64_t N, void* out, int32_t out_dtype, hipStream_t stream) {
  clear_error();
  if (qssm_status st = check(out_dtype, rows, N)) return st;
  if (rows == 0) return QSSM_OK;
  if (!codes || !scales || !out) return fail(QSSM_ERR_INVALID_ARG, "null required pointer");
  if (out_dtype == QSSM_F16) k_state_dequant<true><<<grid_for(rows), kThreads, 0, stream>>>(codes, scales, rows, N, out);
  else k_state_dequant<false><<<grid_for(rows), kThreads, 0, stream>>>(codes, scales, rows, N, out);
  return launch_status("state_dequant");
}
