// W8A8 linear layer: int8 weights x int8 activations on int8 MFMA with int32 accumulation.
//
// Quamba2, abstract: W8A8 blocks, prefill and generation (the in and out projections around the
// recurrence).
//     y[m, n] = bias[n] + fl32(sa[m] sw[n]) * sum_k a[m, k] w[n, k]
// Both operands have k contiguous, which is the operand order of v_mfma_i32_32x32x32_i8: lane l of a
// wave holds row (or column) l % 32 and the 16 consecutive k at 16 (l / 32).
#include <hip/hip_runtime.h>

#include "common.hpp"

using namespace qssm;

namespace {

typedef int v4i __attribute__((ext_vector_type(4)));
typedef int v16i __attribute__((ext_vector_type(16)));

struct GemmParams {
  int64_t M, N, K;
  int32_t per_row, yf16;
  const int8_t* a;
  int64_t as;
  const float* a_scales;
  const int8_t* w;
  int64_t ws;
  const float* w_scales;
  const float* bias;
  void* y;
  int64_t ys;
};

__device__ __forceinline__ float valid_or_zero(float s) { return scale_ok(s) ? s : 0.0f; }

// y[m, n] from the integer sum: one rounding of the sum to fp32 (sums above 2^24), one of the product
// of the scales, one of the fused multiply-add, one more to fp16.
__device__ __forceinline__ void put(const GemmParams& p, int64_t m, int64_t n, int acc, float sa,
                                    float sw, float bn) {
  const float v = fmaf(sa * sw, (float)acc, bn);
  if (p.yf16) reinterpret_cast<__half*>(p.y)[m * p.ys + n] = __float2half_rn(v);
  else reinterpret_cast<float*>(p.y)[m * p.ys + n] = v;
}

// 16 consecutive codes of a row from k on, at any alignment (the hardware takes unaligned 16-byte
// loads); codes at or past K read as 0 without touching memory.
__device__ __forceinline__ uint4 load16(const int8_t* row, int64_t k, int64_t K) {
  uint4 v = make_uint4(0u, 0u, 0u, 0u);
  if (k + 16 <= K) {
    __builtin_memcpy(&v, row + k, 16);
  } else if (k < K) {
    uint32_t w[4] = {0u, 0u, 0u, 0u};
#pragma unroll
    for (int i = 0; i < 16; ++i)
      if (k + i < K) w[i / 4] |= (uint32_t)(uint8_t)row[k + i] << (8 * (i % 4));
    v = make_uint4(w[0], w[1], w[2], w[3]);
  }
  return v;
}

// Any shape and alignment: 128 x 128 tiles of y, K in steps of 64 through LDS (rows padded to 80
// bytes: no bank conflicts), four waves with 64 x 64 each; the next step's global loads are in
// registers during the current step's products. Rows past M or N load a valid row and are not
// stored.
constexpr int kBM = 128, kBN = 128, kBK = 64, kRow = 80;

struct GemmSmem {
  int8_t a[2][kBM * kRow];
  int8_t w[2][kBN * kRow];
};

__global__ __launch_bounds__(256) void k_gemm_w8a8(GemmParams p) {
  __shared__ __align__(16) GemmSmem s;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = uniform(tid >> 6);
  const int wm = wave >> 1, wn = wave & 1, kh = lane >> 5;
  const int64_t m0 = (int64_t)blockIdx.y * kBM, n0 = (int64_t)blockIdx.x * kBN;
  const int64_t nk = (p.K + kBK - 1) / kBK;

  v16i acc[2][2];
#pragma unroll
  for (int mt = 0; mt < 2; ++mt)
#pragma unroll
    for (int nt = 0; nt < 2; ++nt) acc[mt][nt] = v16i{};

  // thread t loads the 32 bytes at 32 (t % 2) of row t / 2 of both tiles
  const int row = tid >> 1, half = (tid & 1) * 32;
  const int8_t* ar = p.a + min(m0 + row, p.M - 1) * p.as;
  const int8_t* wr = p.w + min(n0 + row, p.N - 1) * p.ws;
  uint4 ra[2], rw[2];
  auto load = [&](int64_t kt) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      ra[i] = load16(ar, kt * kBK + half + 16 * i, p.K);
      rw[i] = load16(wr, kt * kBK + half + 16 * i, p.K);
    }
  };
  auto store = [&](int buf) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      *reinterpret_cast<uint4*>(s.a[buf] + row * kRow + half + 16 * i) = ra[i];
      *reinterpret_cast<uint4*>(s.w[buf] + row * kRow + half + 16 * i) = rw[i];
    }
  };
  if (nk > 0) {
    load(0);
    store(0);
  }
  __syncthreads();
  for (int64_t kt = 0; kt < nk; ++kt) {
    const int buf = (int)(kt & 1);
    if (kt + 1 < nk) load(kt + 1);
#pragma unroll
    for (int ks = 0; ks < kBK / 32; ++ks) {
      v4i av[2], bv[2];
#pragma unroll
      for (int mt = 0; mt < 2; ++mt)
        av[mt] = *reinterpret_cast<const v4i*>(s.a[buf] + (wm * 64 + mt * 32 + (lane & 31)) * kRow + ks * 32 + 16 * kh);
#pragma unroll
      for (int nt = 0; nt < 2; ++nt)
        bv[nt] = *reinterpret_cast<const v4i*>(s.w[buf] + (wn * 64 + nt * 32 + (lane & 31)) * kRow + ks * 32 + 16 * kh);
#pragma unroll
      for (int mt = 0; mt < 2; ++mt)
#pragma unroll
        for (int nt = 0; nt < 2; ++nt)
          acc[mt][nt] = __builtin_amdgcn_mfma_i32_32x32x32_i8(av[mt], bv[nt], acc[mt][nt], 0, 0, 0);
    }
    if (kt + 1 < nk) {
      store(buf ^ 1);
      __syncthreads();
    }
  }

  // register r of a tile holds row 8 (r / 4) + 4 (l / 32) + r % 4, column l % 32
#pragma unroll
  for (int nt = 0; nt < 2; ++nt) {
    const int64_t n = n0 + wn * 64 + nt * 32 + (lane & 31);
    if (n >= p.N) continue;
    const float sw = valid_or_zero(p.w_scales[n]), bn = p.bias ? p.bias[n] : 0.0f;
#pragma unroll
    for (int mt = 0; mt < 2; ++mt)
#pragma unroll
      for (int r = 0; r < 16; ++r) {
        const int64_t m = m0 + wm * 64 + mt * 32 + 8 * (r / 4) + 4 * kh + (r % 4);
        if (m < p.M) put(p, m, n, acc[mt][nt][r], valid_or_zero(p.a_scales[p.per_row ? m : 0]), sw, bn);
      }
  }
}

}  // namespace

extern "C" qssm_status qssm_gemm_w8a8(const qssm_gemm_w8a8_args* a, hipStream_t stream) {
  clear_error();
  if (!a) return fail(QSSM_ERR_INVALID_ARG, "args is null");
  const int64_t M = a->M, N = a->N, K = a->K;
  if (M < 0 || N < 0 || K < 0) return fail(QSSM_ERR_INVALID_ARG, "negative extent");
  if (a->y_dtype != QSSM_F32 && a->y_dtype != QSSM_F16)
    return fail(QSSM_ERR_INVALID_ARG, "y_dtype must be QSSM_F32 or QSSM_F16");
  if (K > 131071) return fail(QSSM_ERR_UNSUPPORTED, "K above 131071 (int32 sums)");
  if (a->a_stride < K || a->w_stride < K || a->y_stride < N)
    return fail(QSSM_ERR_INVALID_ARG, "a row stride is smaller than the row");
  const int64_t lim = (int64_t)1 << 40;  // row offsets stay far inside 64 bits
  if (a->a_stride > lim || a->w_stride > lim || a->y_stride > lim || M > 0x7fffffff || N > 0x7fffffff)
    return fail(QSSM_ERR_UNSUPPORTED, "M or N above 2^31 - 1 or a stride above 2^40");
  if (M == 0 || N == 0) return QSSM_OK;
  if (!a->a_scales || !a->w_scales || !a->y || (K > 0 && (!a->a || !a->w)))
    return fail(QSSM_ERR_INVALID_ARG, "null required pointer");
  if (((uintptr_t)a->y) % (a->y_dtype == QSSM_F16 ? 2 : 4) != 0)
    return fail(QSSM_ERR_INVALID_ARG, "y is not aligned to its type");
  const int64_t gx = cdiv(N, kBN), gy = cdiv(M, kBM);
  if (gy > 65535) return fail(QSSM_ERR_UNSUPPORTED, "M above 65535 * 128");
  const GemmParams p{M, N, K, a->a_per_row != 0, a->y_dtype == QSSM_F16, a->a, a->a_stride, a->a_scales,
                     a->w, a->w_stride, a->w_scales, a->bias, a->y, a->y_stride};
  k_gemm_w8a8<<<dim3((unsigned)gx, (unsigned)gy), 256, 0, stream>>>(p);
  return launch_status("gemm_w8a8");
}
