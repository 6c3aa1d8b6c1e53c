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
// 16384 rows of 8192 fp16 channels to int8: 132 us, 3.1 TB/s, of which the issue of vector instructions takes 112 (6.4e7
// slots of four cycles over 1024 SIMDs): 28 an element, half of them silu and the code; to fp16 144 us, 3.7 TB/s.
// 256 single rows of 10240 channels to fp16: 10 us, 4.2 TB/s.
// Channels of a lane, 8 / 4 / 2 / 1: 220 / 172 / 137 / 168 us for the 16384 rows, 19 / 13.4 / 10.4 / 12.8 for the 256 (more
// of them leave too few waves, one alone has 2-byte accesses); rows ahead, 4 / 8 / 16: 142 / 137 / 152.
//
// In-place states: the strip that holds a sequence's first row reads its old state and writes its new one (the
// last W - 1 inputs, most often far behind the strip), and also computes the W - 1 rows that need the old
// one, past its own end if need be; the strip behind begins that much later.
#include <hip/hip_runtime.h>

#include <type_traits>

#include "causal_conv_forms.hpp"
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

// v / (1 + e^-v). Where e^-v overflows (v < -88) the simple form gives -0 for a value of at most 5.3e-37, which fp16 and
// int8 outputs round to 0 as well (the least valid scale is 2^-100); the other form keeps it, by e^-|v| <= 1.
template <bool SIMPLE>
__device__ __forceinline__ float silu_fast(float v) {
  if (SIMPLE) return v * __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(v * -1.44269504f));
  const float e = __builtin_amdgcn_exp2f(-fabsf(v) * 1.44269504f);
  const float r = __builtin_amdgcn_rcpf(1.0f + e);
  return v * (v < 0.0f ? e * r : r);
}

// x, and the compiler does not know that: no fp64 copies of the weights are kept in registers for the rare path.
__device__ __forceinline__ float opaque(float x) {
  asm volatile("" : "+v"(x));
  return x;
}

// The larger of two |x| as they lie in memory, by their bits (a NaN is the largest), two of fp16 at a time.
__device__ __forceinline__ uint32_t larger(uint32_t a, uint32_t b) { return max(a & 0x7fffffffu, b & 0x7fffffffu); }
typedef unsigned short v2u __attribute__((ext_vector_type(2)));
__device__ __forceinline__ v2u larger(v2u a, v2u b) {
  const v2u m = {0x7fff, 0x7fff};
  return __builtin_elementwise_max((v2u)(a & m), (v2u)(b & m));
}

template <int VEC, int W, typename X, typename Y>
struct Lane {
  static constexpr bool kI8 = std::is_same_v<Y, int8_t>;
  const ConvParams& p;
  int c;  // the lane's first channel
  float w[VEC][W], bias[VEC];
  // int8: the reciprocal of the scale (0: no valid one), and what a code's distance from the nearest half-integer loses
  // for each unit of |x|, and without any
  float rc[VEC], loss[VEC], room[VEC];
  const X* x;
  Y* y;

  __device__ __forceinline__ Lane(const ConvParams& q, int channel) : p(q), c(channel) {
    x = reinterpret_cast<const X*>(p.x) + c;
    y = reinterpret_cast<Y*>(p.y) + c;
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
      float sum = 0.0f;
#pragma unroll
      for (int k = 0; k < W; ++k) {
        w[i][k] = p.w[(int64_t)(c + i) * W + k];
        sum += fabsf(w[i][k]);
      }
      bias[i] = p.bias ? p.bias[c + i] : 0.0f;
      if constexpr (kI8) {
        rc[i] = recip_or_zero(scale(i));
        constexpr float kSum = 1.13f * (W + 1) * 0x1p-24f;
        loss[i] = -kSum * sum * rc[i];
        room[i] = 0.4999f - kSum * fabsf(bias[i]) * rc[i];
      }
    }
  }

  __device__ __forceinline__ float scale(int i) const { return p.scales[min((int)p.group_of[c + i], p.groups - 1)]; }
  __device__ __forceinline__ bool has(int i) const { return !p.seq.has || p.seq.has[i] != 0; }
  __device__ __forceinline__ Raw<VEC, X> row(int64_t t) const { return load_raw<VEC>(x + t * p.xs); }

  // The largest |x| of each channel over `rows` rows.
  template <int N>
  __device__ __forceinline__ void largest(const Raw<VEC, X> (&r)[N], float (&m)[VEC]) const {
    if constexpr (std::is_same_v<X, uint16_t> && VEC % 2 == 0) {
#pragma unroll
      for (int i = 0; i < VEC; i += 2) {
        v2u a = {0, 0};
#pragma unroll
        for (int k = 0; k < N; ++k) a = larger(a, v2u{r[k].v[i], r[k].v[i + 1]});
        m[i] = as_float((X)a[0]);
        m[i + 1] = as_float((X)a[1]);
      }
    } else {
#pragma unroll
      for (int i = 0; i < VEC; ++i) {
        uint32_t a = 0;
#pragma unroll
        for (int k = 0; k < N; ++k) a = max(a, std::is_same_v<X, uint16_t> ? r[k].v[i] & 0x7fffu : r[k].v[i] & 0x7fffffffu);
        m[i] = as_float((X)a);
      }
    }
  }

  // Output row t of the W input rows from r[0] on (the oldest first); limit: room less the loss at the largest |x|.
  //
  // int8 codes are those of the value in fp64, rounded once to fp32. The fp32 value decides where it is sure to give the
  // same: its sum is off by at most W 2^-24 (|bias| + sum |w x|), which silu passes on by at most 1.1 times, and the value
  // by (6 + |v|) 2^-23 of itself (the exponent's rounding |v| 2^-23, exponential and reciprocal 2^-23 each, four
  // roundings of 2^-24, the definition's rounding and the quotient's). A code is sure where the quotient is nearer
  // than 1/2 less these to a whole number. Lanes where it is not (1 in ~4000 for ordinary inputs) take the fp64 path.
  __device__ __forceinline__ void put(int64_t t, const Raw<VEC, X>* r, const float (&limit)[VEC]) const {
    constexpr bool kSimple = kI8 || std::is_same_v<Y, uint16_t>;
    constexpr float kMagic = 12582912.0f;  // 1.5 2^23: the sum with it holds the rounded value in its low bits
    Raw<VEC, Y> o;
    bool sure[VEC], all = true;
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
      float v = bias[i];
#pragma unroll
      for (int k = 0; k < W; ++k) v = fmaf(w[i][k], as_float(r[k].v[i]), v);
      const float z = p.silu ? silu_fast<kSimple>(v) : v;
      if constexpr (kI8) {
        const float f = z * rc[i], fc = __builtin_amdgcn_fmed3f(f, -128.0f, 127.0f);
        const float m = fc + kMagic, d = fc - (m - kMagic);
        // (not less: a NaN is not sure either)
        sure[i] = fabsf(d) < fmaf(-fabsf(f), fmaf(fabsf(v), 0x1p-23f, 6.0f * 0x1p-23f), limit[i]);
        all &= sure[i];
        o.v[i] = (int8_t)__float_as_uint(m);
      } else if constexpr (std::is_same_v<Y, uint16_t>) {
        o.v[i] = __half_as_ushort(__float2half_rn(z));
      } else {
        o.v[i] = __float_as_uint(z);
      }
    }
    if constexpr (kI8) {
      if (!all) {
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
          if (sure[i]) continue;
          double v = opaque(bias[i]);
#pragma unroll
          for (int k = 0; k < W; ++k) v = fma((double)opaque(w[i][k]), (double)as_float(r[k].v[i]), v);
          if (p.silu) v = v / (1.0 + exp(-v));
          o.v[i] = quant8((float)v, scale(i));
        }
      }
    }
    store_raw<VEC>(y + t * p.ys, o);
  }

  __device__ __forceinline__ void limits(const float (&m)[VEC], float (&limit)[VEC]) const {
#pragma unroll
    for (int i = 0; i < VEC; ++i) limit[i] = fmaf(loss[i], m[i], room[i]);
  }

  // A sequence's initial rows, the oldest first.
  __device__ __forceinline__ void initial(int64_t slot, bool has, Raw<VEC, X>* r) const {
    const bool given = p.state && slot >= 0 && has;
    const X* at = reinterpret_cast<const X*>(p.state) + slot * (W - 1) * p.C + c;
#pragma unroll
    for (int j = 0; j < W - 1; ++j) r[j] = given ? load_raw<VEC>(at + (int64_t)j * p.C) : Raw<VEC, X>{};
  }

  // The state behind a sequence of `len` rows from `begin` on: its last W - 1 rows, the initial ones before its first.
  __device__ __forceinline__ void final(int64_t slot, int64_t begin, int len, const Raw<VEC, X>* init) const {
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
};


template <int VEC, int W, typename X, typename Y>
__global__ __launch_bounds__(256) void k_causal_conv(ConvParams p) {
  constexpr int kAhead = VEC == 2 ? 8 : 4;  // rows loaded ahead
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
  using L = Lane<VEC, W, X, Y>;
  const L ln(p, c);
  // the rows before t, then kAhead rows from t on
  Raw<VEC, X> win[W - 1 + kAhead], next[kAhead];
  // sequence s begins at row t
  const auto enter = [&](Raw<VEC, X>* before) {
    const int64_t slot = seq_slot(sq, s);
    ln.initial(slot, ln.has(s), before);
    ln.final(slot, begin, end - begin, before);
    te = max(te, (int)min((int64_t)begin + W - 1, (int64_t)end));
  };
  if (t == begin) {
    enter(win);
  } else {
    // (at least W - 1 rows behind begin; offsets out of order can name a sequence that is not, and no row lies before row 0)
#pragma unroll
    for (int j = 0; j < W - 1; ++j) win[j] = t < end ? ln.row(max(t - (W - 1) + j, 0)) : Raw<VEC, X>{};
  }
  const auto load = [&](int64_t from) {
#pragma unroll
    for (int u = 0; u < kAhead; ++u)
      if (from + u < last) next[u] = ln.row(from + u);
  };
  load(t);
  while (t < te) {
#pragma unroll
    for (int u = 0; u < kAhead; ++u) win[W - 1 + u] = next[u];
    const bool ahead = t + kAhead < te;
    if (ahead) load((int64_t)t + kAhead);
    float limit[VEC], m[VEC];
    const bool whole = t + kAhead <= min(te, end);
    if (whole) {
      if constexpr (L::kI8) {
        ln.largest(win, m);
        ln.limits(m, limit);
      }
#pragma unroll
      for (int u = 0; u < kAhead; ++u) ln.put((int64_t)t + u, win + u, limit);
#pragma unroll
      for (int j = 0; j < W - 1; ++j) win[j] = win[kAhead + j];
    } else {
      // rows of more than one sequence, or the strip's last
#pragma unroll 1
      for (int u = 0; u < kAhead && t + u < te; ++u) {
        while (t + u >= end && s + 1 < sq.nseq) {  // the next sequence, past those without rows
          ++s;
          begin = end;
          end = uniform(max(seq_end(sq, s, seq_begin(sq, s)), begin));
          if (t + u < end) enter(win);
        }
        Raw<VEC, X> r[W];
#pragma unroll
        for (int j = 0; j < W - 1; ++j) r[j] = win[j];
        r[W - 1] = ln.row(t + u);
        if constexpr (L::kI8) {
          ln.largest(r, m);
          ln.limits(m, limit);
        }
        ln.put((int64_t)t + u, r, limit);
#pragma unroll
        for (int j = 0; j < W - 1; ++j) win[j] = r[j + 1];
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
  using L = Lane<VEC, W, X, Y>;
  const L ln(p, (int)(id % per) * VEC);
  Raw<VEC, X> r[W];
  const int64_t slot = seq_slot(p.seq, i);
  ln.initial(slot, ln.has(i), r);
  r[W - 1] = ln.row(i);
  float limit[VEC], m[VEC];
  if constexpr (L::kI8) {
    ln.largest(r, m);
    ln.limits(m, limit);
  }
  ln.put(i, r, limit);
  if (p.state_out && slot >= 0) {
    X* at = reinterpret_cast<X*>(p.state_out) + slot * (W - 1) * p.C + ln.c;
#pragma unroll
    for (int k = 0; k < W - 1; ++k) store_raw<VEC>(at + (int64_t)k * p.C, r[k + 1]);
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
  const int64_t strip = qssm_conv::strip_rows(p.seq.tokens, p.cblocks);
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
  return p.C % 2 == 0 ? launch<2, W, X, Y>(p, step, stream) : launch<1, W, X, Y>(p, step, stream);
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
