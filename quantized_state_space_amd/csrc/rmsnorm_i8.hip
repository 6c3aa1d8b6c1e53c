// RMS norm with an int8 output: the residual stream's addition or Mamba2's gate, the norm over one
// or several channel groups, and the quantization of a W8A8 / W4A8 projection's input, in one pass.
//
//     h = round(x + residual)      t = fl32(h * silu(gate))      r_g = fl32((sum t^2 / Dg + eps)^-1/2)
//     v = fl32(fl32(t r_g) w)      s = row_scale(absmax v) or static      q = quant8(v, s)
//
// One workgroup owns one row and holds it in registers from the loads to the codes (VPT vectors of
// VEC channels per thread, vector v of thread i at channel (v T + i) VEC), so every tensor is read
// and written once: the floor is the bytes. Two workgroup reductions join the threads: the sum of
// squares and the largest |v|. The sum is taken in fp64 (squares of fp32 values are exact there), so
// that r, and with it every code, does not depend on the order of the sum beyond ~2^-50; silu is
// evaluated in fp64 to the same end.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "common.hpp"

using namespace qssm;

namespace {

constexpr int kMaxThreads = 1024;
constexpr int kMaxWaves = kMaxThreads / 64;
constexpr int64_t kMaxDimNarrow = 8192;  // VEC = 1: 8 channels per thread (16 with many long rows)
constexpr int64_t kMaxDimWide = 32768;   // VEC = 8: 4 vectors of 8 per thread

struct NormParams {
  int64_t M;
  int32_t D, Dg, Gn, dynamic;
  uint32_t inv_dg;  // ceil(2^32 / Dg): c / Dg is the high word of c * inv_dg for c, Dg <= 32768
  const void* x;
  const void* res;
  void* res_out;
  const void* gate;
  int64_t xs, rs, ros, gs, qs;
  const float* w;
  float eps;
  float* scales;
  int8_t* q;
};

typedef int v2i __attribute__((ext_vector_type(2)));
typedef int v4i __attribute__((ext_vector_type(4)));
constexpr int kBufferWord3 = 0x00020000;  // buffer resource word 3 for raw 32-bit access (gfx9)

// Raw buffer over `n` bytes of a row (n = 0: nothing). Loads past them give 0 and stores past them are
// dropped, so a thread's accesses need no branches and all its loads are in flight together (with a
// branch around each vector's loads they waited one after the other: 8192 x 5001 fp16, 141 us for 82).
__device__ __forceinline__ __amdgpu_buffer_rsrc_t row_rsrc(const void* p, int64_t byte, int n) {
  const char* q = reinterpret_cast<const char*>(p) + (p ? byte : 0);
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<char*>(q), (short)0, p ? n : 0, kBufferWord3);
}

// VEC consecutive elements (16-byte aligned when VEC = 8) as they lie in memory
template <int VEC, bool F16>
struct Raw {
  v4i w[VEC == 8 ? (F16 ? 1 : 2) : 1];
};

template <int VEC, bool F16>
__device__ __forceinline__ Raw<VEC, F16> load_raw(__amdgpu_buffer_rsrc_t r, int c) {
  Raw<VEC, F16> o;
  if constexpr (VEC == 8) {
    o.w[0] = __builtin_bit_cast(v4i, __builtin_amdgcn_raw_buffer_load_b128(r, c * (F16 ? 2 : 4), 0, 0));
    if constexpr (!F16) o.w[1] = __builtin_bit_cast(v4i, __builtin_amdgcn_raw_buffer_load_b128(r, c * 4 + 16, 0, 0));
  } else if constexpr (F16) {
    o.w[0][0] = (int)(unsigned short)__builtin_amdgcn_raw_buffer_load_b16(r, c * 2, 0, 0);
  } else {
    o.w[0][0] = (int)__builtin_amdgcn_raw_buffer_load_b32(r, c * 4, 0, 0);
  }
  return o;
}

template <int VEC, bool F16>
__device__ __forceinline__ void to_float(const Raw<VEC, F16>& r, float (&o)[VEC]) {
#pragma unroll
  for (int k = 0; k < VEC; ++k) {
    if constexpr (F16) {
      const uint32_t w = (uint32_t)r.w[0][k / 2];
      o[k] = __half2float(__ushort_as_half((unsigned short)(k % 2 ? w >> 16 : w & 0xFFFFu)));
    } else {
      o[k] = __builtin_bit_cast(float, (int)r.w[k / 4][k % 4]);
    }
  }
}

// Rounds v to the stream's type and stores it; v becomes the stored value.
template <int VEC, bool F16>
__device__ __forceinline__ void round_store(__amdgpu_buffer_rsrc_t r, int c, float (&v)[VEC]) {
  if constexpr (F16) {
    uint32_t w[(VEC + 1) / 2] = {};
#pragma unroll
    for (int k = 0; k < VEC; ++k) {
      const __half h = __float2half_rn(v[k]);
      v[k] = __half2float(h);
      w[k / 2] |= (uint32_t)__half_as_ushort(h) << (16 * (k % 2));
    }
    if constexpr (VEC == 8) __builtin_amdgcn_raw_buffer_store_b128(v4i{(int)w[0], (int)w[1], (int)w[2], (int)w[3]}, r, c * 2, 0, 0);
    else __builtin_amdgcn_raw_buffer_store_b16((unsigned short)w[0], r, c * 2, 0, 0);
  } else {
    if constexpr (VEC == 8) {
      const auto bits = [&](int k) { return __builtin_bit_cast(int, v[k]); };
      __builtin_amdgcn_raw_buffer_store_b128(v4i{bits(0), bits(1), bits(2), bits(3)}, r, c * 4, 0, 0);
      __builtin_amdgcn_raw_buffer_store_b128(v4i{bits(4), bits(5), bits(6), bits(7)}, r, c * 4 + 16, 0, 0);
    } else {
      __builtin_amdgcn_raw_buffer_store_b32(__builtin_bit_cast(int, v[0]), r, c * 4, 0, 0);
    }
  }
}

// silu(z) = z / (1 + e^-z), in fp64 and rounded once to fp32. With y = -z / ln2 = n + f, |f| <= 1/2:
// e^-z = 2^n p(f), p the polynomial of degree 9 with the least largest relative error against 2^f
// (1.4e-14; coefficients by Remez exchange in 50 digits). Adding 1.5 * 2^52 rounds y to n, which is
// then in the low word. The exponent's argument is clamped where silu rounds to z or to -0 either way:
// an fp16 gate's n at 200 (65504 * 2^-200), an fp32 gate's z at 200 (the largest number * e^-200 is
// 2^-160, below half the least denormal 2^-149). An infinite gate gives an infinity or a NaN, which
// leave its group's codes at 0. One Newton step takes the reciprocal to ~2^-46.
template <bool F16>
__device__ __forceinline__ float silu_f64(float z) {
  constexpr double kLog2e = 1.4426950408889634, kMagic = 6755399441055744.0;
  const double x = -(double)(F16 ? z : __builtin_amdgcn_fmed3f(z, -200.0f, 200.0f));
  const double t = fma(x, kLog2e, kMagic);
  const double f = fma(x, kLog2e, -(t - kMagic));
  double e = 0x1.b3f42432927dap-24;
  e = fma(e, f, 0x1.63edf11a7df52p-20);
  e = fma(e, f, 0x1.ffce245dbe28dp-17);
  e = fma(e, f, 0x1.43088fca865dap-13);
  e = fma(e, f, 0x1.5d87fd9013458p-10);
  e = fma(e, f, 0x1.3b2ab72a10a42p-7);
  e = fma(e, f, 0x1.c6b08d70d1ff5p-5);
  e = fma(e, f, 0x1.ebfbdff81570dp-3);
  e = fma(e, f, 0x1.62e42fefa3752p-1);
  e = fma(e, f, 0x1.0000000000039p+0);
  int n = (int)(uint32_t)__builtin_bit_cast(uint64_t, t);
  if (F16) n = min(max(n, -200), 200);
  const uint64_t bits = __builtin_bit_cast(uint64_t, e);
  const uint32_t hi = (uint32_t)(bits >> 32) + ((uint32_t)n << 20);
  const double d = 1.0 + __builtin_bit_cast(double, ((uint64_t)hi << 32) | (uint32_t)bits);
  double r = __builtin_amdgcn_rcp(d);
  r = fma(fma(-d, r, 1.0), r, r);
  return (float)((F16 ? -x : (double)z) * r);
}

__device__ __forceinline__ float group_r(double sum, int Dg, float eps) {
  return (float)(1.0 / sqrt(sum / (double)Dg + (double)eps));
}

// RES: 0 no residual stream, 1 fp16, 2 fp32. GATE: 0 none, 1 fp16, 2 fp32.
template <int VEC, int VPT, bool XF16, int RES, int GATE>
__global__ __launch_bounds__(kMaxThreads) void k_rmsnorm_i8(NormParams p) {
  extern __shared__ __align__(16) unsigned char smem[];  // several groups: one partial per vector
  __shared__ double red_sum[kMaxWaves];
  __shared__ float red_max[kMaxWaves];
  const int64_t row = (int64_t)blockIdx.y * gridDim.x + blockIdx.x;
  if (row >= p.M) return;  // grid padding (the whole workgroup)
  const int tid = threadIdx.x, T = blockDim.x, lane = tid & 63, wave = tid >> 6, nw = T >> 6;

  constexpr int kXB = XF16 ? 2 : 4, kRB = RES == 1 ? 2 : 4, kZB = GATE == 1 ? 2 : 4;
  const __amdgpu_buffer_rsrc_t rx = row_rsrc(p.x, row * p.xs * kXB, p.D * kXB);
  Raw<VEC, XF16> xr[VPT];
  Raw<VEC, RES == 1> rr[RES ? VPT : 1];
  Raw<VEC, GATE == 1> zr[GATE ? VPT : 1];
#pragma unroll
  for (int v = 0; v < VPT; ++v) xr[v] = load_raw<VEC, XF16>(rx, (v * T + tid) * VEC);
  if constexpr (RES != 0) {
    const __amdgpu_buffer_rsrc_t r = row_rsrc(p.res, row * p.rs * kRB, p.D * kRB);
#pragma unroll
    for (int v = 0; v < VPT; ++v) rr[v] = load_raw<VEC, RES == 1>(r, (v * T + tid) * VEC);
  }
  if constexpr (GATE != 0) {
    const __amdgpu_buffer_rsrc_t r = row_rsrc(p.gate, row * p.gs * kZB, p.D * kZB);
#pragma unroll
    for (int v = 0; v < VPT; ++v) zr[v] = load_raw<VEC, GATE == 1>(r, (v * T + tid) * VEC);
  }

  // the weight too, ahead of the reduction: 8192 x 5001 with an fp32 stream 129 -> 113 us, 1111 x 1543
  // 8.1 -> 7.3, aligned rows alike
  const __amdgpu_buffer_rsrc_t rw = row_rsrc(p.w, 0, p.D * 4);
  Raw<VEC, false> wr[VPT];
#pragma unroll
  for (int v = 0; v < VPT; ++v) wr[v] = load_raw<VEC, false>(rw, (v * T + tid) * VEC);

  // channels past D hold 0 from here on (or NaN after r, which no reduction counts)
  float t[VPT][VEC];
  double sum = 0.0;
  [[maybe_unused]] const __amdgpu_buffer_rsrc_t ro = row_rsrc(p.res_out, row * p.ros * kRB, p.D * kRB);
#pragma unroll
  for (int v = 0; v < VPT; ++v) {
    const int c = (v * T + tid) * VEC;
    to_float<VEC, XF16>(xr[v], t[v]);
    if constexpr (RES != 0) {
      if (p.res) {
        float o[VEC];
        to_float<VEC, RES == 1>(rr[v], o);
#pragma unroll
        for (int k = 0; k < VEC; ++k) t[v][k] += o[k];
      }
      // res_out may be res: each element was read above by the thread that writes it here
      round_store<VEC, RES == 1>(ro, c, t[v]);
    }
    if constexpr (GATE != 0) {
      float z[VEC];
      to_float<VEC, GATE == 1>(zr[v], z);
#pragma unroll
      for (int k = 0; k < VEC; ++k) t[v][k] *= silu_f64<GATE == 1>(z[k]);
    }
    double part = 0.0;
#pragma unroll
    for (int k = 0; k < VEC; ++k) part = fma((double)t[v][k], (double)t[v][k], part);
    if (p.Gn > 1) {
      // a vector lies in one group (Dg % VEC == 0)
      if (c < p.D) {
        if constexpr (VEC == 1) reinterpret_cast<float*>(smem)[c] = t[v][0];
        else reinterpret_cast<double*>(smem)[c / VEC] = part;
      }
    } else {
      sum += part;
    }
  }

  float r1 = 0.0f;
  if (p.Gn > 1) {
    // wave k sums the groups k, k + nw, ... and leaves r in the group's first slot
    __syncthreads();
    const int per = p.Dg / VEC;
    for (int g = wave; g < p.Gn; g += nw) {
      double a = 0.0;
      for (int i = g * per + lane; i < (g + 1) * per; i += 64) {
        if constexpr (VEC == 1) {
          const double u = (double)reinterpret_cast<const float*>(smem)[i];
          a = fma(u, u, a);
        } else {
          a += reinterpret_cast<const double*>(smem)[i];
        }
      }
#pragma unroll
      for (int off = 32; off > 0; off >>= 1) a += __shfl_xor(a, off, 64);
      // every lane's reads precede: the shuffles wait for all of them (r as the double's low word: the
      // array keeps one type)
      if (lane == 0) {
        const float r = group_r(a, p.Dg, p.eps);
        if constexpr (VEC == 1) reinterpret_cast<float*>(smem)[g * per] = r;
        else reinterpret_cast<double*>(smem)[g * per] = __builtin_bit_cast(double, (uint64_t)__builtin_bit_cast(uint32_t, r));
      }
    }
    __syncthreads();
  } else {
#pragma unroll
    for (int off = 32; off > 0; off >>= 1) sum += __shfl_xor(sum, off, 64);
    if (lane == 0) red_sum[wave] = sum;
    __syncthreads();
    double a = 0.0;
    for (int k = 0; k < nw; ++k) a += red_sum[k];
    r1 = group_r(a, p.Dg, p.eps);
  }

  float amax = 0.0f;
#pragma unroll
  for (int v = 0; v < VPT; ++v) {
    const int c = (v * T + tid) * VEC;
    float r = r1;
    if (p.Gn > 1) {
      const int cc = min(c, p.D - VEC);  // (past D: any group's)
      const int g = p.Dg > 1 ? (int)__umulhi((uint32_t)cc, p.inv_dg) : cc, per = p.Dg / VEC;
      if constexpr (VEC == 1) r = reinterpret_cast<const float*>(smem)[g * per];
      else r = __builtin_bit_cast(float, (uint32_t)__builtin_bit_cast(uint64_t, reinterpret_cast<const double*>(smem)[g * per]));
    }
#pragma unroll
    for (int k = 0; k < VEC; ++k) t[v][k] *= r;
    if (p.w) {
      float w[VEC];
      to_float<VEC, false>(wr[v], w);
#pragma unroll
      for (int k = 0; k < VEC; ++k) t[v][k] *= w[k];
    }
#pragma unroll
    for (int k = 0; k < VEC; ++k) amax = fmaxf(amax, fabsf(t[v][k]));  // a NaN does not count
  }

  float s;
  if (p.dynamic) {
    if (amax > 3.402823466e38f) {  // infinities do not count: the largest of the others
      amax = 0.0f;
#pragma unroll
      for (int v = 0; v < VPT; ++v)
#pragma unroll
        for (int k = 0; k < VEC; ++k) amax = fmaxf(amax, finite_abs(t[v][k]));
    }
#pragma unroll
    for (int off = 32; off > 0; off >>= 1) amax = fmaxf(amax, __shfl_xor(amax, off, 64));
    if (lane == 0) red_max[wave] = amax;
    __syncthreads();
    for (int k = 0; k < nw; ++k) amax = fmaxf(amax, red_max[k]);
    s = row_scale(amax);
    if (tid == 0) p.scales[row] = s;
  } else {
    s = p.scales[0];
  }

  const __amdgpu_buffer_rsrc_t rq = row_rsrc(p.q, row * p.qs, p.D);
  if constexpr (VEC == 8) {
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
      uint32_t w[2];
      quant_row<false, 8>(t[v], s, w);
      __builtin_amdgcn_raw_buffer_store_b64(v2i{(int)w[0], (int)w[1]}, rq, (v * T + tid) * 8, 0, 0);
    }
  } else {
    constexpr int kN = (VPT + 3) / 4 * 4;
    float u[kN];
    uint32_t w[kN / 4];
#pragma unroll
    for (int v = 0; v < kN; ++v) u[v] = v < VPT ? t[v < VPT ? v : 0][0] : 0.0f;
    quant_row<false, kN>(u, s, w);
#pragma unroll
    for (int v = 0; v < VPT; ++v)
      __builtin_amdgcn_raw_buffer_store_b8((unsigned char)(w[v / 4] >> (8 * (v % 4))), rq, v * T + tid, 0, 0);
  }
}

template <int VEC, int VPT, bool XF16>
void launch_vpt(const NormParams& p, int res, int gate, dim3 rows, int threads, hipStream_t st) {
  size_t smem = 0;
  if (p.Gn > 1) smem = VEC == 1 ? (size_t)p.D * 4 : (size_t)(p.D / VEC) * 8;
  if (gate == 1) k_rmsnorm_i8<VEC, VPT, XF16, 0, 1><<<rows, threads, smem, st>>>(p);
  else if (gate == 2) k_rmsnorm_i8<VEC, VPT, XF16, 0, 2><<<rows, threads, smem, st>>>(p);
  else if (res == 1) k_rmsnorm_i8<VEC, VPT, XF16, 1, 0><<<rows, threads, smem, st>>>(p);
  else if (res == 2) k_rmsnorm_i8<VEC, VPT, XF16, 2, 0><<<rows, threads, smem, st>>>(p);
  else k_rmsnorm_i8<VEC, VPT, XF16, 0, 0><<<rows, threads, smem, st>>>(p);
}

template <int VEC, bool XF16>
void launch_vec(const NormParams& p, int res, int gate, hipStream_t st) {
  const int64_t nvec = p.D / VEC;
  // Few rows: as many threads as the row feeds (latency). Many: smaller workgroups, of which more run
  // at once and cover each other's reductions. Wide, up to 256 / 512 threads: 16384 x 8192 gated 196 /
  // 203 us, 16384 x 4096 with a stream 132 / 128. Narrow, up to 64 / 256: 16000 x 130 11.7 / 21.7,
  // 8192 x 1001 21.9 / 23.8; 8 / 16 channels per thread: 8192 x 5001 fp16 82 / 54, fp32 84 / 71 (with
  // an fp32 stream 123 / 130), 8192 x 8001 fp16 with a stream 139 / 122, but 1111 x 1543 8.1 / 10.0.
  const bool few = p.M < 512;
  const int cap = few ? kMaxThreads : (VEC == 1 ? 64 : gate ? 256 : 512);
  const int most = VEC == 8 ? 4 : (few || p.D <= 2048 ? 8 : 16);  // vectors per thread
  const int threads = (int)std::min<int64_t>(cdiv(nvec, 64) * 64, std::max<int64_t>(cap, cdiv(cdiv(nvec, most), 64) * 64));
  const int64_t vpt = cdiv(nvec, threads);
  // a grid dimension holds fewer than 2^32 threads
  const int64_t gx = std::min<int64_t>(p.M, (int64_t)1 << 21);
  const dim3 grid((unsigned)gx, (unsigned)cdiv(p.M, gx));
  if (vpt == 1) return launch_vpt<VEC, 1, XF16>(p, res, gate, grid, threads, st);
  if (vpt == 2) return launch_vpt<VEC, 2, XF16>(p, res, gate, grid, threads, st);
  if (vpt <= 4) return launch_vpt<VEC, 4, XF16>(p, res, gate, grid, threads, st);
  if constexpr (VEC == 1) {
    if (vpt <= 8) return launch_vpt<VEC, 8, XF16>(p, res, gate, grid, threads, st);
    launch_vpt<VEC, 16, XF16>(p, res, gate, grid, threads, st);
  }
}

bool dtype_ok(int32_t t) { return t == QSSM_F32 || t == QSSM_F16; }

// A workgroup reads its row before it writes any of it, and another's row may be read after: an output is
// apart from every other tensor, or residual_out is, element by element, residual or x.
qssm_status check_apart(const qssm_rmsnorm_args* a) {
  const int64_t M = a->rows, D = a->dim;
  const int64_t xb = a->x_dtype == QSSM_F16 ? 2 : 4, rb = a->residual_dtype == QSSM_F16 ? 2 : 4,
                zb = a->gate_dtype == QSSM_F16 ? 2 : 4;
  const auto rows = [&](const void* t, int64_t stride, int64_t size) {  // (a null tensor's stride is not read)
    return t ? Span{t, M, stride * size, D * size} : Span{};
  };
  const Span x = rows(a->x, a->x_stride, xb), r = rows(a->residual, a->residual_stride, rb),
             ro = rows(a->residual_out, a->residual_out_stride, rb), z = rows(a->gate, a->gate_stride, zb),
             q = rows(a->q, a->q_stride, 1), w = flat(a->weight, D * 4), s = flat(a->scales, a->compute_scales ? M * 4 : 4);
  const auto itself = [&](const Span& t) { return ro.p == t.p && ro.width == t.width && (M == 1 || ro.stride == t.stride); };
  if (overlap(q, x) || overlap(q, r) || overlap(q, ro) || overlap(q, z) || overlap(q, w) || overlap(q, s))
    return fail(QSSM_ERR_INVALID_ARG, "q overlaps another tensor");
  if ((!itself(x) && overlap(ro, x)) || (!itself(r) && overlap(ro, r)) || overlap(ro, w) || overlap(ro, s))
    return fail(QSSM_ERR_INVALID_ARG, "residual_out overlaps another tensor (it may be residual or x itself)");
  if (a->compute_scales && (overlap(s, x) || overlap(s, r) || overlap(s, z) || overlap(s, w)))
    return fail(QSSM_ERR_INVALID_ARG, "scales overlaps another tensor");
  return QSSM_OK;
}

}  // namespace

extern "C" qssm_status qssm_rmsnorm_i8(const qssm_rmsnorm_args* a, hipStream_t stream) {
  clear_error();
  if (!a) return fail(QSSM_ERR_INVALID_ARG, "args is null");
  const int64_t M = a->rows, D = a->dim;
  if (M < 0 || D < 1) return fail(QSSM_ERR_INVALID_ARG, "rows must be >= 0 and dim >= 1");
  if (a->norm_groups < 1 || D % a->norm_groups != 0)
    return fail(QSSM_ERR_INVALID_ARG, "norm_groups must divide dim");
  if (!dtype_ok(a->x_dtype)) return fail(QSSM_ERR_INVALID_ARG, "x_dtype must be QSSM_F32 or QSSM_F16");
  const bool stream_on = a->residual || a->residual_out;
  if (stream_on && !dtype_ok(a->residual_dtype))
    return fail(QSSM_ERR_INVALID_ARG, "residual_dtype must be QSSM_F32 or QSSM_F16");
  if (a->gate && !dtype_ok(a->gate_dtype))
    return fail(QSSM_ERR_INVALID_ARG, "gate_dtype must be QSSM_F32 or QSSM_F16");
  if (a->gate && stream_on)
    return fail(QSSM_ERR_UNSUPPORTED, "a gate together with a residual stream");
  if (!(a->eps >= 0.0f) || a->eps > 3.402823466e38f)
    return fail(QSSM_ERR_INVALID_ARG, "eps must be finite and >= 0");
  // row offsets in bytes stay inside 64 bits
  const int64_t lim = std::min((int64_t)1 << 40, ((int64_t)1 << 58) / std::max<int64_t>(M, 1));
  if (a->x_stride < D || a->q_stride < D || (a->residual && a->residual_stride < D) ||
      (a->residual_out && a->residual_out_stride < D) || (a->gate && a->gate_stride < D))
    return fail(QSSM_ERR_INVALID_ARG, "a row stride is smaller than dim");
  if (a->x_stride > lim || a->q_stride > lim || (a->residual && a->residual_stride > lim) ||
      (a->residual_out && a->residual_out_stride > lim) || (a->gate && a->gate_stride > lim) ||
      M > 0x7fffffff)
    return fail(QSSM_ERR_UNSUPPORTED, "rows above 2^31 - 1, a stride above 2^40 or rows * stride above 2^58");
  if (a->residual && a->residual == a->residual_out && a->residual_stride != a->residual_out_stride)
    return fail(QSSM_ERR_INVALID_ARG, "residual_out == residual needs one stride");
  const int64_t Dg = D / a->norm_groups;
  uint64_t a16 = (uint64_t)(uintptr_t)a->x | (uintptr_t)a->residual | (uintptr_t)a->residual_out |
                 (uintptr_t)a->gate | (uintptr_t)a->weight;
  int64_t strides = a->x_stride | a->q_stride;
  if (a->residual) strides |= a->residual_stride;
  if (a->residual_out) strides |= a->residual_out_stride;
  if (a->gate) strides |= a->gate_stride;
  const bool wide = Dg % 8 == 0 && strides % 8 == 0 && a16 % 16 == 0 && (uintptr_t)a->q % 8 == 0;
  if (D > (wide ? kMaxDimWide : kMaxDimNarrow))
    return fail(QSSM_ERR_UNSUPPORTED, "dim above 8192 (32768 with aligned rows and groups)");
  if (M == 0) return QSSM_OK;
  if (!a->x || !a->scales || !a->q) return fail(QSSM_ERR_INVALID_ARG, "null required pointer");
  const auto off_type = [](const void* t, int32_t type) { return (uintptr_t)t % (type == QSSM_F16 ? 2 : 4) != 0; };
  if (off_type(a->x, a->x_dtype) || off_type(a->weight, QSSM_F32) || off_type(a->scales, QSSM_F32) ||
      (stream_on && (off_type(a->residual, a->residual_dtype) || off_type(a->residual_out, a->residual_dtype))) ||
      (a->gate && off_type(a->gate, a->gate_dtype)))
    return fail(QSSM_ERR_INVALID_ARG, "a tensor is not aligned to its type");
  if (qssm_status st = check_apart(a)) return st;
  NormParams p{M, (int32_t)D, (int32_t)Dg, a->norm_groups, a->compute_scales != 0,
               Dg > 1 ? (uint32_t)((((uint64_t)1 << 32) + Dg - 1) / Dg) : 0u, a->x, a->residual, a->residual_out,
               a->gate, a->x_stride, a->residual_stride, a->residual_out_stride, a->gate_stride,
               a->q_stride, a->weight, a->eps, a->scales, a->q};
  const int res = !stream_on ? 0 : (a->residual_dtype == QSSM_F16 ? 1 : 2);
  const int gate = !a->gate ? 0 : (a->gate_dtype == QSSM_F16 ? 1 : 2);
  const bool xf16 = a->x_dtype == QSSM_F16;
  if (wide) {
    if (xf16) launch_vec<8, true>(p, res, gate, stream);
    else launch_vec<8, false>(p, res, gate, stream);
  } else {
    if (xf16) launch_vec<1, true>(p, res, gate, stream);
    else launch_vec<1, false>(p, res, gate, stream);
  }
  return launch_status("rmsnorm_i8");
}
