// a14: fused decode state update (generation stage), Mamba2-shaped.
//
// Quamba2, abstract: W8A8 generation for the Mamba2 backbone. One token per sequence: x, B and C
// are quantized with static scales (the a1/a2 rule), then for every state element of head h
//     state = exp(delta A_h) state + delta xh[p] Bh[n],    y[p] = sum_n Ch[n] state + D_h xh[p]
//
// The state (P x N per (b, h), fp32 or fp16) is the only large operand: the kernel is one
// streaming read-modify-write pass over it. A workgroup owns one (b, h) state tile: it quantizes
// and dequantizes the P x values and the N B/C values of its group into LDS once, then each thread
// updates 4 (fp32) or 8 (fp16) consecutive states per 16-byte access with fully coalesced wave
// accesses, and the readout sum over n is a shuffle reduction among the lanes sharing a row.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "common.hpp"

using namespace qssm;

namespace {

constexpr int kThreads = 256;
constexpr int kMaxRows = 256;  // rows of an int8 state tile

struct UpdParams {
  int64_t B, nh, P, N;
  int32_t Gbc, hpg, gs, G;
  const float* x;
  const uint8_t* x_group_of;
  const float* x_scales;
  const float* Bm;
  const float* Cm;
  const float* B_scales;
  const float* C_scales;
  const float* delta;
  const float* A;
  const float* Dskip;
  void* state;
  void* y;
  int8_t* xq_out;
  int8_t* Bq_out;
  int8_t* Cq_out;
  int32_t yi8, Gy;            // int8 output, number of output groups
  const uint8_t* y_group_of;  // int8 output: [nh * P]
  const float* y_scales;      // int8 output: [Gy]
  const float* y_bias;        // int8 output: [nh * P] or NULL
};

// Quantizes and dequantizes the P x values of (b, h) = bh and the N B/C values of its group into
// LDS, publishing the codes where asked, and waits for the workgroup.
__device__ __forceinline__ void stage_inputs(const UpdParams& p, int64_t bh, float* xs, float* bs,
                                             float* cs) {
  const int64_t b = bh / p.nh, h = bh % p.nh;
  const int64_t g = h / p.hpg;
  const int ngs = (int)(p.N / p.gs);
  const bool write_bc = (h % p.hpg) == 0;  // one head per group publishes the B/C codes

  for (int64_t k = threadIdx.x; k < p.P; k += kThreads) {
    const int64_t i = bh * p.P + k;
    const float s = p.x_scales[min((int)p.x_group_of[h * p.P + k], p.G - 1)];
    const int8_t q = quant8(p.x[i], s);
    if (p.xq_out) p.xq_out[i] = q;
    xs[k] = scale_ok(s) ? (float)q * s : 0.0f;
  }
  for (int64_t n = threadIdx.x; n < p.N; n += kThreads) {
    const int64_t i = (b * p.Gbc + g) * p.N + n;
    const float sb = p.B_scales[g * ngs + n / p.gs];
    const float sc = p.C_scales[g * ngs + n / p.gs];
    const int8_t qb = quant8(p.Bm[i], sb), qc = quant8(p.Cm[i], sc);
    if (write_bc) {
      if (p.Bq_out) p.Bq_out[i] = qb;
      if (p.Cq_out) p.Cq_out[i] = qc;
    }
    bs[n] = scale_ok(sb) ? (float)qb * sb : 0.0f;
    cs[n] = scale_ok(sc) ? (float)qc * sc : 0.0f;
  }
  __syncthreads();
}

// y[i] of channel ch (= h * P + p), fp32 or int8 codes. Persistent int8 output: fl32(y + correction term), the exact rule
// with the channel's static output scale.
__device__ __forceinline__ void store_y(const UpdParams& p, int64_t i, int64_t ch, float yv) {
  if (p.yi8) {
    const float sy = p.y_scales[min((int)p.y_group_of[ch], p.Gy - 1)];
    const float yb = p.y_bias ? p.y_bias[ch] : 0.0f;
    reinterpret_cast<int8_t*>(p.y)[i] = quant8_r(yv + yb, sy, recip_or_zero(sy));
  } else {
    reinterpret_cast<float*>(p.y)[i] = yv;
  }
}

// CH consecutive states per thread access: 4 for fp32 (16 bytes), 8 for fp16 (16 bytes).
// R = N / CH lanes share one state row.
template <int F16, int R>
__global__ __launch_bounds__(kThreads) void k_state_update(UpdParams p) {
  constexpr int CH = F16 ? 8 : 4;
  extern __shared__ float smem[];
  float* xs = smem;                    // [P], padded to a multiple of 4
  float* bs = xs + ((p.P + 3) & ~3);   // [N], 16-byte aligned (N % 4 == 0)
  float* cs = bs + p.N;                // [N]

  const int64_t bh = blockIdx.x;  // b * nh + h
  const int64_t h = bh % p.nh;
  stage_inputs(p, bh, xs, bs, cs);

  const float dt = p.delta[bh];
  const float dA = expf(dt * p.A[h]);
  const float Dh = p.Dskip ? p.Dskip[h] : 0.0f;
  const int64_t nch = p.N / CH;
  const int64_t total = p.P * nch;  // CH-element chunks of the tile
  const int lane = threadIdx.x & 63;

  for (int64_t base = 0; base < total; base += kThreads) {
    const int64_t f = base + threadIdx.x;
    const bool on = f < total;
    const int64_t row = on ? f / nch : 0;
    const int64_t n0 = on ? (f - row * nch) * CH : 0;
    float s[CH];
#pragma unroll
    for (int k = 0; k < CH; ++k) s[k] = 0.0f;
    uint4 raw = make_uint4(0u, 0u, 0u, 0u);
    if (on) raw = reinterpret_cast<const uint4*>(p.state)[bh * total + f];
    if (F16) {
      const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const __half2 v = *reinterpret_cast<const __half2*>(&w[k]);
        s[2 * k] = __low2float(v);
        s[2 * k + 1] = __high2float(v);
      }
    } else {
      s[0] = __uint_as_float(raw.x); s[1] = __uint_as_float(raw.y);
      s[2] = __uint_as_float(raw.z); s[3] = __uint_as_float(raw.w);
    }
    const float dtx = dt * xs[row];
    // B and C of the CH states in 16-byte LDS reads (n0 and the N-float arrays are 4-aligned)
    float bv[CH], cv[CH];
#pragma unroll
    for (int k4 = 0; k4 < CH / 4; ++k4) {
      const float4 b4 = *reinterpret_cast<const float4*>(bs + n0 + 4 * k4);
      const float4 c4 = *reinterpret_cast<const float4*>(cs + n0 + 4 * k4);
      bv[4 * k4] = b4.x; bv[4 * k4 + 1] = b4.y; bv[4 * k4 + 2] = b4.z; bv[4 * k4 + 3] = b4.w;
      cv[4 * k4] = c4.x; cv[4 * k4 + 1] = c4.y; cv[4 * k4 + 2] = c4.z; cv[4 * k4 + 3] = c4.w;
    }
    float yp = 0.0f;
#pragma unroll
    for (int k = 0; k < CH; ++k) {
      s[k] = fmaf(dA, s[k], dtx * bv[k]);
      yp = fmaf(cv[k], s[k], yp);
    }
    if (on) {
      uint4 out;
      if (F16) {
        uint32_t w[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const __half2 v = __floats2half2_rn(s[2 * k], s[2 * k + 1]);
          w[k] = *reinterpret_cast<const uint32_t*>(&v);
        }
        out = make_uint4(w[0], w[1], w[2], w[3]);
      } else {
        out = make_uint4(__float_as_uint(s[0]), __float_as_uint(s[1]), __float_as_uint(s[2]),
                         __float_as_uint(s[3]));
      }
      reinterpret_cast<uint4*>(p.state)[bh * total + f] = out;
    }
    // rows occupy R consecutive lanes (R divides 64 and kThreads): reduce within them
#pragma unroll
    for (int off = R / 2; off > 0; off >>= 1) yp += __shfl_xor(yp, off, 64);
    if (on && (lane % R) == 0) {
      store_y(p, bh * p.P + row, h * p.P + row, fmaf(Dh, xs[row], yp));
    }
  }
}

// int8 state. A workgroup owns a tile of consecutive rows (h, p) of one (b, B/C group): it quantizes
// the group's B and C once for all of them and leaves dA, delta x and D x of each row in LDS. R = N / 16
// lanes share a row, 16 codes (16 bytes) each; a thread's 16 states n are the same in every row, so B and C stay
// in its registers. The row's readout and new absmax are DPP reductions over those lanes, and the new
// state waits in registers for its scale: the codes are read and written once. The loads of the first
// rows are issued before the inputs are quantized, whose chain of dependent loads they cover, and
// from then on one batch ahead.
struct StateI8 {
  const int8_t* in;
  const float* s_in;
  int8_t* out;
  float* s_out;
  int64_t tiles;  // of `rows` rows per (b, group)
  int32_t rows;
};

constexpr float kMaxInRange = 0x1.fcp+106f;  // 127 * 2^100: the scale of a larger absmax is clamped

template <int R>
__device__ __forceinline__ float row_sum(float x) {
  if constexpr (R >= 2) x += dpp_partner<1>(x);
  if constexpr (R >= 4) x += dpp_partner<2>(x);
  if constexpr (R >= 8) x += dpp_partner<4>(x);
  if constexpr (R >= 16) x += dpp_partner<8>(x);
  return x;
}

template <int R>
__device__ __forceinline__ float row_max(float x) {
  if constexpr (R >= 2) x = fmaxf(x, dpp_partner<1>(x));
  if constexpr (R >= 4) x = fmaxf(x, dpp_partner<2>(x));
  if constexpr (R >= 8) x = fmaxf(x, dpp_partner<4>(x));
  if constexpr (R >= 16) x = fmaxf(x, dpp_partner<8>(x));
  return x;
}

template <int R>
__global__ __launch_bounds__(kThreads) void k_state_update_i8(UpdParams p, StateI8 st) {
  // products and sums round where the definition says (the new codes are fixed bit for bit); the fused ones are
  // written as such
#pragma clang fp contract(off)
  constexpr int N = 16 * R, kPass = kThreads / R, kBatch = 2;  // rows per pass, passes in flight
  __shared__ __align__(16) float bs[N], cs[N];
  __shared__ __align__(16) float4 rowc[kMaxRows];
  const int tid = threadIdx.x;
  const int64_t id = (int64_t)blockIdx.y * gridDim.x + blockIdx.x;
  const int64_t bg = id / st.tiles;  // b * Gbc + g
  if (bg >= p.B * p.Gbc) return;     // grid padding (the whole workgroup)
  const int64_t tile = id % st.tiles;
  const int64_t b = bg / p.Gbc, g = bg % p.Gbc;
  const int64_t grows = p.hpg * p.P;  // rows of the group
  const int64_t r0 = tile * st.rows;
  const int n_rows = (int)min((int64_t)st.rows, grows - r0);
  const int64_t at0 = bg * grows + r0;  // first row in the state ([B, nh, P] = [B, Gbc, hpg P])

  const int sub = tid % R, n0 = 16 * sub, lrow = tid / R;
  uint4 raw[kBatch];
  float s_in[kBatch];
  auto load = [&](int base) {
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const int row = base + i * kPass + lrow;
      raw[i] = make_uint4(0u, 0u, 0u, 0u);
      s_in[i] = 0.0f;
      if (row < n_rows) {
        raw[i] = *reinterpret_cast<const uint4*>(st.in + (at0 + row) * N + n0);
        s_in[i] = st.s_in[at0 + row];
      }
    }
  };
  load(0);

  for (int k = tid; k < n_rows; k += kThreads) {
    const int64_t ch = g * grows + r0 + k;  // h * P + p
    const int64_t h = ch / p.P;
    const float s = p.x_scales[min((int)p.x_group_of[ch], p.G - 1)];
    const int8_t q = quant8(p.x[at0 + k], s);
    if (p.xq_out) p.xq_out[at0 + k] = q;
    const float x = scale_ok(s) ? (float)q * s : 0.0f;
    const float dt = p.delta[b * p.nh + h];
    rowc[k] = make_float4((float)exp((double)(dt * p.A[h])), dt * x, (p.Dskip ? p.Dskip[h] : 0.0f) * x, 0.0f);
  }
  const int ngs = N / p.gs;
  for (int k = tid; k < 2 * N; k += kThreads) {
    const int n = k % N;
    const int64_t i = bg * N + n;
    const float s = (k < N ? p.B_scales : p.C_scales)[g * ngs + n / p.gs];
    const int8_t q = quant8((k < N ? p.Bm : p.Cm)[i], s);
    int8_t* out = k < N ? p.Bq_out : p.Cq_out;
    if (tile == 0 && out) out[i] = q;
    (k < N ? bs : cs)[n] = scale_ok(s) ? (float)q * s : 0.0f;
  }
  __syncthreads();
  float bv[16], cv[16];
#pragma unroll
  for (int k = 0; k < 16; k += 4) {
    const float4 b4 = *reinterpret_cast<const float4*>(bs + n0 + k), c4 = *reinterpret_cast<const float4*>(cs + n0 + k);
    bv[k] = b4.x; bv[k + 1] = b4.y; bv[k + 2] = b4.z; bv[k + 3] = b4.w;
    cv[k] = c4.x; cv[k + 1] = c4.y; cv[k + 2] = c4.z; cv[k + 3] = c4.w;
  }

  for (int base = 0; base < n_rows; base += kBatch * kPass) {
    uint4 now[kBatch];
    float s_now[kBatch];
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      now[i] = raw[i];
      s_now[i] = s_in[i];
    }
    if (base + kBatch * kPass < n_rows) load(base + kBatch * kPass);
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const int row = base + i * kPass + lrow;
      const bool on = row < n_rows;
      const float4 rc = rowc[on ? row : 0];
      const float keep = scale_ok(s_now[i]) ? rc.x * s_now[i] : 0.0f;
      const uint32_t w[4] = {now[i].x, now[i].y, now[i].z, now[i].w};
      float v[16];
      float yp = 0.0f, amax = 0.0f;
#pragma unroll
      for (int k = 0; k < 16; ++k) {
        const float q = (float)(int8_t)(w[k / 4] >> (8 * (k % 4)));
        v[k] = fmaf(keep, q, rc.y * bv[k]);
        yp = fmaf(cv[k], v[k], yp);
        amax = fmaxf(amax, fabsf(v[k]));
      }
      yp = row_sum<R>(yp);
      amax = row_max<R>(amax);
      uint32_t o[4];
      float sn;
      if (amax <= kMaxInRange && yp == yp) {
        // every value is finite (a NaN or an infinity would show in yp or in amax)
        sn = row_scale(amax);
        quant_row<true, 16>(v, sn, o);
      } else {
        amax = 0.0f;
#pragma unroll
        for (int k = 0; k < 16; ++k) amax = fmaxf(amax, finite_abs(v[k]));
        sn = row_scale(row_max<R>(amax));
        quant_row<false, 16>(v, sn, o);
      }
      if (on) {
        *reinterpret_cast<uint4*>(st.out + (at0 + row) * N + n0) = make_uint4(o[0], o[1], o[2], o[3]);
        if (sub == 0) {
          st.s_out[at0 + row] = sn;
          store_y(p, at0 + row, g * grows + r0 + row, rc.z + yp);
        }
      }
    }
  }
}

template <int R>
void launch_i8(const UpdParams& p, StateI8 st, hipStream_t stream) {
  const int64_t grows = p.hpg * p.P;
  // Large tiles share one quantization of B and C; small ones keep a small batch spread over the GPU.
  st.rows = p.B * p.nh * p.P >= kMaxRows * 2048 ? kMaxRows : 64;
  st.tiles = cdiv(grows, st.rows);
  // a grid dimension holds fewer than 2^32 threads
  const int64_t n = p.B * p.Gbc * st.tiles, gx = std::min<int64_t>(n, (int64_t)1 << 23);
  k_state_update_i8<R><<<dim3((unsigned)gx, (unsigned)cdiv(n, gx)), kThreads, 0, stream>>>(p, st);
}

template <int R>
qssm_status launch_r(const UpdParams& p, int f16, hipStream_t st) {
  const size_t smem = (size_t)(((p.P + 3) & ~3) + 2 * p.N) * sizeof(float);
  const unsigned grid = (unsigned)(p.B * p.nh);
  if (f16) {
    if constexpr (R % 2 == 0) k_state_update<1, R / 2><<<grid, kThreads, smem, st>>>(p);
  } else {
    k_state_update<0, R><<<grid, kThreads, smem, st>>>(p);
  }
  return launch_status("state_update");
}

// Checks shared by the state types: before (shapes and types) and after (pointers and sizes) the
// checks of the state's own type.
qssm_status check_shape(const qssm_update_args* a) {
  const int64_t B = a->batch, nh = a->nheads, P = a->headdim, N = a->dstate;
  if (B < 0 || nh < 1 || P < 1 || N < 1) return fail(QSSM_ERR_INVALID_ARG, "bad shape");
  if (a->ngroups < 1 || nh % a->ngroups != 0)
    return fail(QSSM_ERR_INVALID_ARG, "ngroups must divide nheads");
  if (a->bc_group_size < 1 || N % a->bc_group_size != 0)
    return fail(QSSM_ERR_INVALID_ARG, "bc_group_size must divide dstate");
  if (a->x_groups < 1 || a->x_groups > 256) return fail(QSSM_ERR_INVALID_ARG, "x_groups not in 1..256");
  if (a->y_dtype != QSSM_F32 && a->y_dtype != QSSM_I8)
    return fail(QSSM_ERR_INVALID_ARG, "y_dtype must be QSSM_F32 or QSSM_I8");
  if (a->y_dtype == QSSM_I8) {
    if (a->y_groups < 1 || a->y_groups > 256)
      return fail(QSSM_ERR_INVALID_ARG, "y_groups not in 1..256");
    if (!a->y_group_of || !a->y_scales)
      return fail(QSSM_ERR_INVALID_ARG, "QSSM_I8 output needs y_group_of and y_scales");
  }
  return QSSM_OK;
}

qssm_status check_rest(const qssm_update_args* a) {
  const int64_t B = a->batch, nh = a->nheads;
  if (!a->x || !a->x_group_of || !a->x_scales || !a->B || !a->C || !a->B_scales || !a->C_scales ||
      !a->delta || !a->A || !a->state || !a->y)
    return fail(QSSM_ERR_INVALID_ARG, "null required pointer");
  if ((uintptr_t)a->state % 16 != 0) return fail(QSSM_ERR_INVALID_ARG, "state must be 16-byte aligned");
  if (B * nh > 0x7fffffffLL) return fail(QSSM_ERR_INVALID_ARG, "batch * nheads too large");
  return QSSM_OK;
}

qssm_status check_headdim(const qssm_update_args* a) {
  const int64_t P = a->headdim, N = a->dstate;
  if ((((P + 3) & ~3) + 2 * N) * 4 > 64 * 1024) return fail(QSSM_ERR_UNSUPPORTED, "headdim too large");
  return QSSM_OK;
}

UpdParams params_of(const qssm_update_args* a) {
  const int64_t B = a->batch, nh = a->nheads, P = a->headdim, N = a->dstate;
  return UpdParams{B, nh, P, N, a->ngroups, (int32_t)(nh / a->ngroups), a->bc_group_size, a->x_groups, a->x,
              a->x_group_of, a->x_scales, a->B, a->C, a->B_scales, a->C_scales, a->delta, a->A,
              a->Dskip, a->state, a->y, a->xq_out, a->Bq_out, a->Cq_out,
              a->y_dtype == QSSM_I8, a->y_dtype == QSSM_I8 ? a->y_groups : 1, a->y_group_of,
              a->y_scales, a->y_bias};
}

}  // namespace

extern "C" qssm_status qssm_state_update(const qssm_update_args* a, hipStream_t stream) {
  clear_error();
  if (!a) return fail(QSSM_ERR_INVALID_ARG, "args is null");
  if (a->state_dtype != QSSM_F32 && a->state_dtype != QSSM_F16)
    return fail(QSSM_ERR_INVALID_ARG, "state_dtype must be QSSM_F32 or QSSM_F16");
  if (qssm_status st = check_shape(a)) return st;
  const int64_t N = a->dstate;
  const int64_t R = N / 4;
  if (N % 4 != 0 || !(R == 1 || R == 2 || R == 4 || R == 8 || R == 16 || R == 32 || R == 64))
    return fail(QSSM_ERR_UNSUPPORTED, "dstate must be 4 * 2^k with 4 <= dstate <= 256");
  if (a->state_dtype == QSSM_F16 && N < 8)
    return fail(QSSM_ERR_UNSUPPORTED, "an fp16 state needs dstate >= 8");
  if (qssm_status st = check_headdim(a)) return st;
  if (a->batch == 0) return QSSM_OK;
  if (qssm_status st = check_rest(a)) return st;
  const UpdParams p = params_of(a);
  const int f16 = a->state_dtype == QSSM_F16;
  switch (R) {
    case 1: return launch_r<1>(p, f16, stream);
    case 2: return launch_r<2>(p, f16, stream);
    case 4: return launch_r<4>(p, f16, stream);
    case 8: return launch_r<8>(p, f16, stream);
    case 16: return launch_r<16>(p, f16, stream);
    case 32: return launch_r<32>(p, f16, stream);
    default: return launch_r<64>(p, f16, stream);
  }
}

extern "C" qssm_status qssm_state_update_i8(const qssm_update_args* a, const int8_t* state_in,
                                            const float* scales_in, float* state_scales,
                                            hipStream_t stream) {
  clear_error();
  if (!a) return fail(QSSM_ERR_INVALID_ARG, "args is null");
  if (a->state_dtype != QSSM_I8) return fail(QSSM_ERR_INVALID_ARG, "state_dtype must be QSSM_I8");
  if (qssm_status st = check_shape(a)) return st;
  const int64_t R = a->dstate / 16;
  if (a->dstate % 16 != 0 || !(R == 1 || R == 2 || R == 4 || R == 8 || R == 16))
    return fail(QSSM_ERR_UNSUPPORTED, "an int8 state needs dstate = 16 * 2^k with 16 <= dstate <= 256");
  if (qssm_status st = check_headdim(a)) return st;
  if ((state_in == nullptr) != (scales_in == nullptr))
    return fail(QSSM_ERR_INVALID_ARG, "state_in and scales_in go together");
  if (a->batch == 0) return QSSM_OK;
  if (!state_scales) return fail(QSSM_ERR_INVALID_ARG, "null required pointer");
  if (qssm_status st = check_rest(a)) return st;
  if ((uintptr_t)state_in % 16 != 0)
    return fail(QSSM_ERR_INVALID_ARG, "state_in must be 16-byte aligned");
  if (a->batch * a->nheads > ((int64_t)1 << 38) / a->headdim)
    return fail(QSSM_ERR_UNSUPPORTED, "batch * nheads * headdim above 2^38");
  // read and written ranges are one or apart: a row half over another's would be read after its write
  const int64_t rows = a->batch * a->nheads * a->headdim;
  const Span q = flat(a->state, rows * a->dstate), s = flat(state_scales, rows * 4),
             qi = flat(state_in, rows * a->dstate), si = flat(scales_in, rows * 4);
  if ((qi.p != q.p && overlap(qi, q)) || (si.p != s.p && overlap(si, s)) || overlap(qi, s) || overlap(si, q))
    return fail(QSSM_ERR_INVALID_ARG, "state_in or scales_in overlaps what is written");
  if (overlap(q, s)) return fail(QSSM_ERR_INVALID_ARG, "state and state_scales overlap");
  const UpdParams p = params_of(a);
  int8_t* out = reinterpret_cast<int8_t*>(a->state);
  const StateI8 st{state_in ? state_in : out, scales_in ? scales_in : state_scales, out, state_scales, 0, 0};
  switch (R) {
    case 1: launch_i8<1>(p, st, stream); break;
    case 2: launch_i8<2>(p, st, stream); break;
    case 4: launch_i8<4>(p, st, stream); break;
    case 8: launch_i8<8>(p, st, stream); break;
    default: launch_i8<16>(p, st, stream); break;
  }
  return launch_status("state_update_i8");
}
