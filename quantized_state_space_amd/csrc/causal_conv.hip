// Short causal convolution over packed sequences, one filter of 2 to 4 taps a channel, with SiLU.
//
// Quamba2, abstract: Mamba1 and Mamba2 blocks, where it stands between the in-projection and the
// recurrence.
//     v[t, c] = bias[c] + sum_k w[c, k] x[t - (W - 1) + k, c],     y = v / (1 + e^-v) or v
//
// Bound by the bytes: x is read once and y written once. A lane owns VEC channels and walks down a strip of
// rows with the last W - 1 inputs in registers, so only the W - 1 rows before a strip are read twice;
// the next rows are loaded while these are computed. A strip that crosses from one sequence into
// the next takes the next one's state where it begins, one branch that is uniform over the wave.
//
// In-place states: the strip that holds a sequence's first row reads its old state and writes its new one (the
// last W - 1 inputs, most often far behind the strip), and also computes the W - 1 rows that need the old
// one, past its own end if need be; the strip behind begins that much later.
#include <hip/hip_runtime.h>

#include <type_traits>

#include "common.hpp"
#include "sequences.hpp"

using namespace qssm;

namespace {

struct ConvParams {
  Seqs seq;
  int32_t C, silu, strip, groups;
  int32_t cblocks, strips;  // channel blocks, strips (behind them: 64 sequences a wave for the empty ones)
  const void* x;
  int64_t xs;
  const float* w;
  const float* bias;
  void* y;
  int64_t ys;
  const void* state;
  void* state_out;
  const uint8_t* group_of;
  const float* scales;
};

// VEC consecutive elements as they lie in memory, at any address that their type allows.
template <int VEC, typename T>
struct Raw {
  T v[VEC];
};

template <int VEC, typename T>
__device__ __forceinline__ Raw<VEC, T> load_raw(const T* p) {
  Raw<VEC, T> r;
  __builtin_memcpy(&r, p, sizeof(r));
  return r;
}

template <int VEC, typename T>
__device__ __forceinline__ void store_raw(T* p, const Raw<VEC, T>& r) {
  __builtin_memcpy(p, &r, sizeof(r));
}

template <typename T>
__device__ __forceinline__ float as_float(T v) {
  if constexpr (std::is_same_v<T, uint16_t>) return __half2float(__ushort_as_half(v));
  else return __uint_as_float(v);
}

// e^-|v| and 1 / (1 + e^-|v|): no overflow on either side.
__device__ __forceinline__ float silu_fast(float v) {
  const float e = __builtin_amdgcn_exp2f(-fabsf(v) * 1.44269504f);
  const float r = __builtin_amdgcn_rcpf(1.0f + e);
  return v * (v < 0.0f ? e * r : r);
}

__device__ __noinline__ float exact_value(const float* w, const float* x, int W, float bias, int silu) {
  double v = bias;
  for (int k = 0; k < W; ++k) v = fma((double)w[k], (double)x[k], v);
  if (silu) v = v / (1.0 + exp(-v));
  return (float)v;
}

// One output row of VEC channels from the W input rows in x (the oldest first).
// int8 codes are those of the value in fp64, rounded once to fp32. The fp32 value decides where it is sure to
// give the same: its sum is off by at most W 2^-24 (|bias| + sum |w x|), which silu passes on by at most
// 1.1 times, and its silu by (8 + |v|) 2^-23 of itself (exponential, reciprocal and two roundings of 2^-23 or
// less, and the exponent's rounding, |v| 2^-24); a code is sure where v / s is further than that from the nearest half-integer.
// Lanes where it is not (~1 in 2000 for ordinary inputs) take the fp64 path.
template <int VEC, int W, typename Y>
__device__ __forceinline__ void put_row(const ConvParams& p, const float (&w)[VEC][W], const float (&bias)[VEC],
                                        const float (&x)[W][VEC], const float (&sc)[VEC], const float (&rc)[VEC],
                                        Y* out) {
  Raw<VEC, Y> o;
#pragma unroll
  for (int c = 0; c < VEC; ++c) {
    float v = bias[c];
#pragma unroll
    for (int k = 0; k < W; ++k) v = fmaf(w[c][k], x[k][c], v);
    float y = p.silu ? silu_fast(v) : v;
    if constexpr (std::is_same_v<Y, int8_t>) {
      float s = fabsf(bias[c]);
#pragma unroll
      for (int k = 0; k < W; ++k) s = fmaf(fabsf(w[c][k]), fabsf(x[k][c]), s);
      const float off = fmaf(s, 1.11f * (W + 1) * 0x1p-24f, fabsf(y) * ((8.0f + fabsf(v)) * 0x1p-23f));
      const float f = __builtin_amdgcn_fmed3f(y * rc[c], -256.0f, 256.0f);
      const float t = rintf(f);
      // (not less: a NaN is not sure either)
      const bool sure = fabsf(f - t) + off * rc[c] * 1.01f < 0.4999f;
      int q = (int)__builtin_amdgcn_fmed3f(t, -128.0f, 127.0f);
      if (!sure) {
        float wk[W], xk[W];
#pragma unroll
        for (int k = 0; k < W; ++k) wk[k] = w[c][k], xk[k] = x[k][c];
        q = quant8(exact_value(wk, xk, W, bias[c], p.silu), sc[c]);
      }
      o.v[c] = (int8_t)(rc[c] != 0.0f ? q : 0);
    } else if constexpr (std::is_same_v<Y, uint16_t>) {
      o.v[c] = __half_as_ushort(__float2half_rn(y));
    } else {
      o.v[c] = __float_as_uint(y);
    }
  }
  store_raw<VEC>(out, o);
}

template <int VEC, int W, typename X, typename Y>
struct Lane {
  const ConvParams& p;
  int c;  // the lane's first channel
  float w[VEC][W], bias[VEC], sc[VEC], rc[VEC];
  const X* x;
  Y* y;

  __device__ __forceinline__ Lane(const ConvParams& q, int channel) : p(q), c(channel) {
    x = reinterpret_cast<const X*>(p.x) + c;
    y = reinterpret_cast<Y*>(p.y) + c;
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
#pragma unroll
      for (int k = 0; k < W; ++k) w[i][k] = p.w[(int64_t)(c + i) * W + k];
      bias[i] = p.bias ? p.bias[c + i] : 0.0f;
      sc[i] = rc[i] = 0.0f;
      if constexpr (std::is_same_v<Y, int8_t>) {
        sc[i] = p.scales[min((int)p.group_of[c + i], p.groups - 1)];
        rc[i] = recip_or_zero(sc[i]);
      }
    }
  }

  __device__ __forceinline__ Raw<VEC, X> row(int64_t t) const { return load_raw<VEC>(x + t * p.xs); }

  // A sequence's initial rows, the oldest first.
  __device__ __forceinline__ void initial(int64_t slot, bool has, Raw<VEC, X> (&r)[W - 1]) const {
    const bool given = p.state && slot >= 0 && has;
    const X* at = reinterpret_cast<const X*>(p.state) + slot * (W - 1) * p.C + c;
#pragma unroll
    for (int j = 0; j < W - 1; ++j) r[j] = given ? load_raw<VEC>(at + (int64_t)j * p.C) : Raw<VEC, X>{};
  }

  // The state behind a sequence of `len` rows from `begin` on: its last W - 1 rows, the initial ones before its first.
  __device__ __forceinline__ void final(int64_t slot, int64_t begin, int len, const Raw<VEC, X> (&init)[W - 1]) const {
    if (!p.state_out || slot < 0) return;
    X* at = reinterpret_cast<X*>(p.state_out) + slot * (W - 1) * p.C + c;
    Raw<VEC, X> r[W - 1];
#pragma unroll
    for (int j = 0; j < W - 1; ++j) {
      const int pos = len - (W - 1) + j;
      if (pos >= 0) {
        r[j] = row(begin + pos);
      } else {
        r[j] = init[W - 2];
#pragma unroll
        for (int k = W - 3; k >= 0; --k)
          if (len + j == k) r[j] = init[k];
      }
    }
#pragma unroll
    for (int j = 0; j < W - 1; ++j) store_raw<VEC>(at + (int64_t)j * p.C, r[j]);
  }

  __device__ __forceinline__ bool has(int i) const { return !p.seq.has || p.seq.has[i] != 0; }
};

constexpr int kAhead = 4;  // rows loaded ahead

template <int VEC, int W, typename X, typename Y>
__global__ __launch_bounds__(256) void k_causal_conv(ConvParams p) {
  const int wave = uniform(threadIdx.x >> 6), lane = threadIdx.x & 63;
  const int cb = blockIdx.x % p.cblocks;
  const int64_t strip = (int64_t)(blockIdx.x / p.cblocks) * 4 + wave;
  const int c = (cb * 64 + lane) * VEC;
  const Seqs& sq = p.seq;
  if (strip >= p.strips) {
    // 64 sequences a wave: those without rows hand their state on
    const int64_t i0 = (strip - p.strips) * 64;
    if (i0 >= sq.nseq) return;
    const int i = (int)min(i0 + lane, (int64_t)sq.nseq - 1), b = seq_begin(sq, i);
    uint64_t empty = __ballot(i0 + lane < sq.nseq && seq_end(sq, i, b) == b);
    if (!empty || c >= p.C) return;
    const Lane<VEC, W, X, Y> ln(p, c);
    for (; empty; empty &= empty - 1) {
      const int e = uniform((int)i0 + __builtin_ctzll(empty));
      Raw<VEC, X> init[W - 1];
      const int64_t slot = seq_slot(sq, e);
      ln.initial(slot, ln.has(e), init);
      ln.final(slot, 0, 0, init);
    }
    return;
  }
  const int t0 = (int)(strip * p.strip);
  const int first = sq.offsets ? seq_begin(sq, 0) : 0;
  const int last = uniform(sq.offsets ? seq_begin(sq, sq.nseq) : sq.tokens);
  int t = uniform(max(t0, first)), te = (int)min((int64_t)t0 + p.strip, (int64_t)last);
  if (t >= te) return;
  int s = sq.offsets ? last_not_above(sq.nseq, t, [&](int i) { return (int64_t)seq_begin(sq, i); }) : uniform(t / sq.each);
  int begin = uniform(seq_begin(sq, s)), end = uniform(seq_end(sq, s, begin));
  if (begin < t0 && t0 - begin < W - 1) t = min(begin + W - 1, end);
  if (c >= p.C) return;
  const Lane<VEC, W, X, Y> ln(p, c);
  float hist[W - 1][VEC];
  const auto keep = [&](const Raw<VEC, X> (&r)[W - 1]) {
#pragma unroll
    for (int j = 0; j < W - 1; ++j)
#pragma unroll
      for (int i = 0; i < VEC; ++i) hist[j][i] = as_float(r[j].v[i]);
  };
  // sequence s begins at row t
  const auto enter = [&]() {
    Raw<VEC, X> init[W - 1];
    const int64_t slot = seq_slot(sq, s);
    ln.initial(slot, ln.has(s), init);
    ln.final(slot, begin, end - begin, init);
    keep(init);
    te = max(te, (int)min((int64_t)begin + W - 1, (int64_t)end));
  };
  if (t == begin) {
    enter();
  } else if (t < end) {
    Raw<VEC, X> before[W - 1];
#pragma unroll
    for (int j = 0; j < W - 1; ++j) before[j] = ln.row(t - (W - 1) + j);
    keep(before);
  }
  Raw<VEC, X> next[kAhead];
  const auto load = [&](int64_t from) {
#pragma unroll
    for (int u = 0; u < kAhead; ++u)
      if (from + u < last) next[u] = ln.row(from + u);
  };
  load(t);
  while (t < te) {
    Raw<VEC, X> now[kAhead];
#pragma unroll
    for (int u = 0; u < kAhead; ++u) now[u] = next[u];
    const bool ahead = t + kAhead < te;
    if (ahead) load((int64_t)t + kAhead);
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      if (t + u < te) {
        while (t + u >= end && s + 1 < sq.nseq) {  // the next sequence, past those without rows
          ++s;
          begin = end;
          end = uniform(max(seq_end(sq, s, seq_begin(sq, s)), begin));
          if (t + u < end) enter();
        }
        float v[W][VEC];
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
#pragma unroll
          for (int k = 0; k < W - 1; ++k) v[k][i] = hist[k][i];
          v[W - 1][i] = as_float(now[u].v[i]);
#pragma unroll
          for (int k = 0; k < W - 1; ++k) hist[k][i] = v[k + 1][i];
        }
        put_row<VEC, W>(p, ln.w, ln.bias, v, ln.sc, ln.rc, ln.y + (int64_t)(t + u) * p.ys);
      }
    }
    if (!ahead && t + kAhead < te) load((int64_t)t + kAhead);  // a sequence that began here goes on past the strip
    t += kAhead;
  }
}

// One row a sequence: a lane owns VEC channels of one sequence, and all its rows are read before any is written.
template <int VEC, int W, typename X, typename Y>
__global__ __launch_bounds__(256) void k_causal_conv_step(ConvParams p) {
  const int64_t id = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int per = p.C / VEC;
  const int i = (int)(id / per);
  if (i >= p.seq.nseq) return;
  const Lane<VEC, W, X, Y> ln(p, (int)(id % per) * VEC);
  Raw<VEC, X> init[W - 1];
  const int64_t slot = seq_slot(p.seq, i);
  ln.initial(slot, ln.has(i), init);
  const Raw<VEC, X> x = ln.row(i);
  float v[W][VEC];
#pragma unroll
  for (int c = 0; c < VEC; ++c) {
#pragma unroll
    for (int k = 0; k < W - 1; ++k) v[k][c] = as_float(init[k].v[c]);
    v[W - 1][c] = as_float(x.v[c]);
  }
  put_row<VEC, W>(p, ln.w, ln.bias, v, ln.sc, ln.rc, ln.y + (int64_t)i * p.ys);
  if (p.state_out && slot >= 0) {
    X* at = reinterpret_cast<X*>(p.state_out) + slot * (W - 1) * p.C + ln.c;
#pragma unroll
    for (int k = 0; k < W - 2; ++k) store_raw<VEC>(at + (int64_t)k * p.C, init[k + 1]);
    store_raw<VEC>(at + (int64_t)(W - 2) * p.C, x);
  }
}

constexpr int64_t kMaxBlocks = ((int64_t)1 << 24) - 1;  // a grid holds fewer than 2^32 threads

template <int VEC, int W, typename X, typename Y>
qssm_status launch(ConvParams p, bool step, hipStream_t stream) {
  if (step) {
    const int64_t blocks = cdiv((int64_t)p.seq.nseq * (p.C / VEC), 256);
    if (blocks > kMaxBlocks) return fail(QSSM_ERR_UNSUPPORTED, "tokens * dim too large");
    k_causal_conv_step<VEC, W, X, Y><<<(unsigned)blocks, 256, 0, stream>>>(p);
    return launch_status("causal_conv");
  }
  p.cblocks = (int32_t)cdiv(p.C, 64 * VEC);
  // strips as long as leaves 8 waves to a SIMD (1024 SIMDs), 8 to 64 rows
  int64_t strip = 64;
  while (strip > 8 && cdiv(p.seq.tokens, strip) * p.cblocks < 8192) strip /= 2;
  p.strip = (int32_t)strip;
  p.strips = (int32_t)cdiv(p.seq.tokens, strip);
  const bool empties = p.state_out && (p.seq.offsets || p.seq.each == 0);
  const int64_t blocks = cdiv(p.strips + (empties ? cdiv(p.seq.nseq, 64) : 0), 4) * p.cblocks;
  if (blocks == 0) return QSSM_OK;
  if (blocks > kMaxBlocks) return fail(QSSM_ERR_UNSUPPORTED, "tokens * dim too large");
  k_causal_conv<VEC, W, X, Y><<<(unsigned)blocks, 256, 0, stream>>>(p);
  return launch_status("causal_conv");
}

template <int W, typename X, typename Y>
qssm_status launch_vec(const ConvParams& p, bool step, hipStream_t stream) {
  return p.C % 8 == 0 ? launch<8, W, X, Y>(p, step, stream) : launch<1, W, X, Y>(p, step, stream);
}

template <int W, typename X>
qssm_status launch_y(const ConvParams& p, int32_t yt, bool step, hipStream_t stream) {
  return yt == QSSM_I8 ? launch_vec<W, X, int8_t>(p, step, stream)
         : yt == QSSM_F16 ? launch_vec<W, X, uint16_t>(p, step, stream)
                          : launch_vec<W, X, uint32_t>(p, step, stream);
}

template <int W>
qssm_status launch_x(const ConvParams& p, int32_t xt, int32_t yt, bool step, hipStream_t stream) {
  return xt == QSSM_F16 ? launch_y<W, uint16_t>(p, yt, step, stream) : launch_y<W, uint32_t>(p, yt, step, stream);
}

}  // namespace

extern "C" qssm_status qssm_causal_conv(const qssm_conv_args* a, hipStream_t stream) {
  clear_error();
  if (!a) return fail(QSSM_ERR_INVALID_ARG, "args is null");
  const int64_t T = a->tokens, C = a->dim, W = a->width;
  if (const qssm_status s = check_seqs(T, C, a->nseq, a->seq_offsets, a->state, a->state_out, a->slots, a->state_slots)) return s;
  if (W < 2 || W > 4) return fail(QSSM_ERR_UNSUPPORTED, "width must be 2, 3 or 4");
  if (a->x_dtype != QSSM_F32 && a->x_dtype != QSSM_F16) return fail(QSSM_ERR_INVALID_ARG, "x_dtype must be QSSM_F32 or QSSM_F16");
  if (a->y_dtype != QSSM_F32 && a->y_dtype != QSSM_F16 && a->y_dtype != QSSM_I8)
    return fail(QSSM_ERR_INVALID_ARG, "y_dtype must be QSSM_F32, QSSM_F16 or QSSM_I8");
  if (a->reserved != 0) return fail(QSSM_ERR_INVALID_ARG, "reserved must be 0");
  const bool i8 = a->y_dtype == QSSM_I8;
  if (i8 && (a->y_groups < 1 || a->y_groups > 256)) return fail(QSSM_ERR_INVALID_ARG, "y_groups must be in 1..256");
  const int64_t sx = type_size(a->x_dtype), sy = type_size(a->y_dtype);
  if (const qssm_status s = check_rows("x", a->x, T, C, a->x_stride, sx)) return s;
  if (const qssm_status s = check_rows("y", a->y, T, C, a->y_stride, sy)) return s;
  if (a->nseq == 0 || C == 0) return QSSM_OK;
  if (!a->weight || (T > 0 && (!a->x || !a->y)) || (i8 && (!a->y_group_of || !a->y_scales)))
    return fail(QSSM_ERR_INVALID_ARG, "null required pointer");
  if (((uintptr_t)a->weight | (uintptr_t)a->bias) % 4 != 0 || (i8 && (uintptr_t)a->y_scales % 4 != 0) ||
      ((uintptr_t)a->state | (uintptr_t)a->state_out) % sx != 0)
    return fail(QSSM_ERR_INVALID_ARG, "weight, bias, y_scales or a state is not aligned to its type");
  if (a->slots > ((int64_t)1 << 58) / (C * 4)) return fail(QSSM_ERR_UNSUPPORTED, "slots * dim above 2^56");
  const int64_t sb = a->slots * (W - 1) * C * sx;
  const Span y{a->y, T, a->y_stride * sy, C * sy}, out = flat(a->state_out, sb);
  const Span in[] = {{a->x, T, a->x_stride * sx, C * sx}, flat(a->weight, C * W * 4), flat(a->bias, C * 4),
                     flat(a->seq_offsets, (a->nseq + 1) * 4), flat(a->state_slots, a->nseq * 4), flat(a->has_state, a->nseq),
                     flat(i8 ? a->y_group_of : nullptr, C), flat(i8 ? a->y_scales : nullptr, a->y_groups * 4)};
  for (const Span& s : in)
    if (overlap(y, s) || overlap(out, s)) return fail(QSSM_ERR_INVALID_ARG, "y or state_out overlaps an input");
  const bool in_place = a->state_out && a->state_out == a->state;
  if (overlap(y, flat(a->state, sb)) || overlap(y, out) || (!in_place && overlap(out, flat(a->state, sb))))
    return fail(QSSM_ERR_INVALID_ARG, "y, state and state_out overlap");
  ConvParams p{};
  p.seq = make_seqs(T, a->nseq, a->seq_offsets, a->state_slots, a->has_state, a->slots);
  p.C = (int32_t)C;
  p.silu = a->silu != 0;
  p.groups = a->y_groups;
  p.x = a->x;
  p.xs = a->x_stride;
  p.w = a->weight;
  p.bias = a->bias;
  p.y = a->y;
  p.ys = a->y_stride;
  p.state = a->state;
  p.state_out = a->state_out;
  p.group_of = a->y_group_of;
  p.scales = a->y_scales;
  const bool step = !a->seq_offsets && T == a->nseq;
  return W == 2   ? launch_x<2>(p, a->x_dtype, a->y_dtype, step, stream)
         : W == 3 ? launch_x<3>(p, a->x_dtype, a->y_dtype, step, stream)
                  : launch_x<4>(p, a->x_dtype, a->y_dtype, step, stream);
}
