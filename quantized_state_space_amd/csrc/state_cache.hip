// int8 recurrent state: rows of N values written as int8 codes with one scale each, and read back.
//
//     s = absmax(finite |h|) fl32(1/127),  q = quant8(h, s)          h' = fl32(s q)
//
// Both are passes bound by the bytes (fp32: 5 B per value each way; 34 us for 2^25 values at the rate of
// a large copy). Rows of up to 256 values in groups of 4: L lanes hold a row, 4 values each, so that a
// wave's loads and stores are whole runs, and kRows rows are in flight per lane; the absmax is a
// reduction over the row's lanes. With one wave per row and single values (the form for other rows)
// 262144 x 128 fp32 takes 92 us to write and 46 us to read back, here 32 and 27 (5.2 TB/s).
#include <hip/hip_runtime.h>

#include <type_traits>

#include "common.hpp"

using namespace qssm;

namespace {

constexpr int kThreads = 256;

// Keeps a product's rounding to fp32 apart from the one to fp16 that follows (the compiler would join
// them in a mixed-precision fma, which rounds once).
__device__ __forceinline__ void round_apart(float& v) { asm("" : "+v"(v)); }

template <bool F16>
__device__ __forceinline__ float load1(const void* h, int64_t i) {
  if constexpr (F16) return __half2float(reinterpret_cast<const __half*>(h)[i]);
  else return reinterpret_cast<const float*>(h)[i];
}

constexpr int kRows = 4;

template <int L>
__device__ __forceinline__ float lanes_max(float a) {
  if constexpr (L >= 2) a = fmaxf(a, dpp_partner<1>(a));
  if constexpr (L >= 4) a = fmaxf(a, dpp_partner<2>(a));
  if constexpr (L >= 8) a = fmaxf(a, dpp_partner<4>(a));
  if constexpr (L >= 16) a = fmaxf(a, dpp_partner<8>(a));
  if constexpr (L >= 32) a = fmaxf(a, __shfl_xor(a, 16, 64));
  if constexpr (L >= 64) a = fmaxf(a, __shfl_xor(a, 32, 64));
  return a;
}

template <int L, bool F16>
__global__ __launch_bounds__(kThreads) void k_state_quant4(const void* h, int64_t rows, int N,
                                                           int8_t* codes, float* scales) {
  const int lane = threadIdx.x & 63, n = 4 * (lane % L);
  const int64_t wave = (int64_t)blockIdx.x * (kThreads / 64) + (threadIdx.x >> 6);
  const int64_t row0 = wave * (kRows * (64 / L)) + lane / L;
  float v[kRows][4];
#pragma unroll
  for (int u = 0; u < kRows; ++u) {
    const int64_t row = row0 + u * (64 / L);
#pragma unroll
    for (int k = 0; k < 4; ++k) v[u][k] = 0.0f;
    if (row < rows && n < N) {
      if constexpr (F16) {
        const uint2 raw = *reinterpret_cast<const uint2*>(reinterpret_cast<const __half*>(h) + row * N + n);
        const __half2 a = *reinterpret_cast<const __half2*>(&raw.x), b = *reinterpret_cast<const __half2*>(&raw.y);
        v[u][0] = __low2float(a); v[u][1] = __high2float(a);
        v[u][2] = __low2float(b); v[u][3] = __high2float(b);
      } else {
        const float4 a = *reinterpret_cast<const float4*>(reinterpret_cast<const float*>(h) + row * N + n);
        v[u][0] = a.x; v[u][1] = a.y; v[u][2] = a.z; v[u][3] = a.w;
      }
    }
  }
#pragma unroll
  for (int u = 0; u < kRows; ++u) {
    const int64_t row = row0 + u * (64 / L);
    float a = 0.0f;
#pragma unroll
    for (int k = 0; k < 4; ++k) a = fmaxf(a, finite_abs(v[u][k]));
    const float s = row_scale(lanes_max<L>(a));
    uint32_t w[1];
    quant_row<false, 4>(v[u], s, w);
    if (row < rows && n < N) {
      *reinterpret_cast<uint32_t*>(codes + row * N + n) = w[0];
      if (n == 0) scales[row] = s;
    }
  }
}

template <int L, bool F16>
__global__ __launch_bounds__(kThreads) void k_state_dequant4(const int8_t* codes, const float* scales,
                                                             int64_t rows, int N, void* out) {
  const int lane = threadIdx.x & 63, n = 4 * (lane % L);
  const int64_t wave = (int64_t)blockIdx.x * (kThreads / 64) + (threadIdx.x >> 6);
  const int64_t row0 = wave * (kRows * (64 / L)) + lane / L;
  uint32_t w[kRows];
  float s[kRows];
#pragma unroll
  for (int u = 0; u < kRows; ++u) {
    const int64_t row = row0 + u * (64 / L);
    w[u] = 0u;
    s[u] = 0.0f;
    if (row < rows && n < N) {
      w[u] = *reinterpret_cast<const uint32_t*>(codes + row * N + n);
      s[u] = scales[row];
    }
  }
#pragma unroll
  for (int u = 0; u < kRows; ++u) {
    const int64_t row = row0 + u * (64 / L);
    if (row >= rows || n >= N) continue;
    const float f = scale_ok(s[u]) ? s[u] : 0.0f;
    float v[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) v[k] = (float)(int8_t)(w[u] >> (8 * k)) * f;
    if constexpr (F16) {
      uint32_t o[2];
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        round_apart(v[2 * k]);
        round_apart(v[2 * k + 1]);
        o[k] = (uint32_t)__half_as_ushort(__float2half_rn(v[2 * k])) |
               ((uint32_t)__half_as_ushort(__float2half_rn(v[2 * k + 1])) << 16);
      }
      *reinterpret_cast<uint2*>(reinterpret_cast<__half*>(out) + row * N + n) = make_uint2(o[0], o[1]);
    } else {
      *reinterpret_cast<float4*>(reinterpret_cast<float*>(out) + row * N + n) = make_float4(v[0], v[1], v[2], v[3]);
    }
  }
}

// Any other row: one wave per row.
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
      if constexpr (F16) round_apart(v);
      if constexpr (F16) reinterpret_cast<__half*>(out)[row * N + n] = __float2half_rn(v);
      else reinterpret_cast<float*>(out)[row * N + n] = v;
    }
  }
}

// The pointers of a call with rows: none null, the values and the scales aligned to their types, no two tensors
// over each other (a row's codes are shorter than its values, so even in place they would lie over other rows').
qssm_status check_tensors(const void* values, int32_t dtype, int64_t rows, int64_t N, const int8_t* codes, const float* scales) {
  if (!values || !codes || !scales) return fail(QSSM_ERR_INVALID_ARG, "null required pointer");
  if ((uintptr_t)values % (dtype == QSSM_F16 ? 2 : 4) != 0 || (uintptr_t)scales % 4 != 0)
    return fail(QSSM_ERR_INVALID_ARG, "a tensor is not aligned to its type");
  const Span v = flat(values, rows * N * (dtype == QSSM_F16 ? 2 : 4)), c = flat(codes, rows * N), s = flat(scales, rows * 4);
  if (overlap(v, c) || overlap(v, s) || overlap(c, s)) return fail(QSSM_ERR_INVALID_ARG, "two of the tensors overlap");
  return QSSM_OK;
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

// Lanes per row of the 4-value forms (a power of two), 0 when the row or its alignment does not allow
// them: values 4 at a time, codes 4 bytes at a time.
int lanes_of(int64_t rows, int64_t N, const void* values, int32_t dtype, const int8_t* codes) {
  if (N % 4 != 0 || N > 256 || (uintptr_t)values % (dtype == QSSM_F16 ? 8 : 16) != 0 || (uintptr_t)codes % 4 != 0)
    return 0;
  int L = 1;
  while (4 * L < N) L *= 2;
  // a grid holds fewer than 2^32 threads
  return cdiv(rows, kRows * (64 / L) * (kThreads / 64)) < ((int64_t)1 << 24) ? L : 0;
}

// Calls f(std::integral_constant L) for L lanes per row.
template <typename F>
void with_lanes(int L, F f) {
  switch (L) {
    case 1: f(std::integral_constant<int, 1>()); break;
    case 2: f(std::integral_constant<int, 2>()); break;
    case 4: f(std::integral_constant<int, 4>()); break;
    case 8: f(std::integral_constant<int, 8>()); break;
    case 16: f(std::integral_constant<int, 16>()); break;
    case 32: f(std::integral_constant<int, 32>()); break;
    default: f(std::integral_constant<int, 64>()); break;
  }
}

}  // namespace

extern "C" qssm_status qssm_state_quant(const void* h, int32_t h_dtype, int64_t rows, int64_t N,
                                        int8_t* codes, float* scales, hipStream_t stream) {
  clear_error();
  if (qssm_status st = check(h_dtype, rows, N)) return st;
  if (rows == 0) return QSSM_OK;
  if (qssm_status st = check_tensors(h, h_dtype, rows, N, codes, scales)) return st;
  const bool f16 = h_dtype == QSSM_F16;
  if (const int L = lanes_of(rows, N, h, h_dtype, codes)) {
    with_lanes(L, [&](auto l) {
      const unsigned grid = (unsigned)cdiv(rows, kRows * (64 / l()) * (kThreads / 64));
      if (f16) k_state_quant4<l(), true><<<grid, kThreads, 0, stream>>>(h, rows, (int)N, codes, scales);
      else k_state_quant4<l(), false><<<grid, kThreads, 0, stream>>>(h, rows, (int)N, codes, scales);
    });
  } else if (f16) {
    k_state_quant<true><<<grid_for(rows), kThreads, 0, stream>>>(h, rows, N, codes, scales);
  } else {
    k_state_quant<false><<<grid_for(rows), kThreads, 0, stream>>>(h, rows, N, codes, scales);
  }
  return launch_status("state_quant");
}

extern "C" qssm_status qssm_state_dequant(const int8_t* codes, const float* scales, int64_t rows,
                                          int64_t N, void* out, int32_t out_dtype, hipStream_t stream) {
  clear_error();
  if (qssm_status st = check(out_dtype, rows, N)) return st;
  if (rows == 0) return QSSM_OK;
  if (qssm_status st = check_tensors(out, out_dtype, rows, N, codes, scales)) return st;
  const bool f16 = out_dtype == QSSM_F16;
  if (const int L = lanes_of(rows, N, out, out_dtype, codes)) {
    with_lanes(L, [&](auto l) {
      const unsigned grid = (unsigned)cdiv(rows, kRows * (64 / l()) * (kThreads / 64));
      if (f16) k_state_dequant4<l(), true><<<grid, kThreads, 0, stream>>>(codes, scales, rows, (int)N, out);
      else k_state_dequant4<l(), false><<<grid, kThreads, 0, stream>>>(codes, scales, rows, (int)N, out);
    });
  } else if (f16) {
    k_state_dequant<true><<<grid_for(rows), kThreads, 0, stream>>>(codes, scales, rows, N, out);
  } else {
    k_state_dequant<false><<<grid_for(rows), kThreads, 0, stream>>>(codes, scales, rows, N, out);
  }
  return launch_status("state_dequant");
}
