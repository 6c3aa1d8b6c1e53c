// Selective scan on unquantized inputs over packed sequences, with softplus, skip and gate.
//
// Quamba2, abstract: the Mamba1 recurrence, prefill and generation.
//     dt = softplus(delta + bias)     h[n] = e^(dt A[n]) h[n] + dt x B[n]     y = (C h + D x) silu(z)
//
// Four neighbouring lanes own a channel, each a quarter of its states (NPL of them, in registers), and a
// workgroup 64 channels of one B/C group. The rows run in batches of four: each lane of a channel loads
// and prepares one row (dt, dt x, and later the gate), the four rows' values are passed around by lane
// permutations, and the four lanes' sums are joined by a transposed reduction that leaves each lane the
// sum of its own row. B and C of 32 rows at a time go through LDS in their own type while the rows before are computed
// (fp16 ones are multiplied as they are, by mixed fused multiply-adds), and the next 32 rows of x, delta and z are in
// registers by then.
//
// Bound by vector instructions: an update takes two products, an exponential (half the rate) and two fused
// multiply-adds, 6 issue slots, of T D N updates. A batch of four rows takes 135 of them for a lane's 16 updates (N 16), 80
// the updates' own. 16 x 1024 rows, 4096 channels, whole: 298 us; the same number of rows in 24 sequences of very
// different lengths: 436 us, about 0.4 of it in the first launch, all of it filled by 2.5e8 issue slots of four cycles over
// 1024 SIMDs (a single pass without cuts: 1.4e8; the updates' slots alone: 175 us); 256 single rows, which the
// bytes of their states bound: 35 us, 4.1 TB/s.
//
// Few sequences with few channels do not fill the chip, so long sequences are cut into pieces (piece_rows()).
// First the pieces but the last run without y, the first from the initial state, the others from zero; then all run in
// full from the state that they fold from the ends before them:
//     h_in[c + 1] = e^(A sum dt over c) h_in[c] + end[c].
// In a packed batch the first pieces, whose state is known, run in full at once (runs_first()).
#include <hip/hip_runtime.h>

#include <algorithm>
#include <initializer_list>
#include <type_traits>

#include "common.hpp"
#include "selective_scan_forms.hpp"
#include "sequences.hpp"

using namespace qssm;

namespace {

struct SscanParams {
  Seqs seq;
  int32_t D, N, G, Dg, per_group;  // Dg = D / G channels in per_group workgroups
  int32_t piece;                   // rows of a piece
  int32_t first;                   // whether the first of several pieces runs in full with the others' ends
  int32_t softplus, yf16, sf16;
  const void *x, *delta, *B, *C, *z;
  int64_t xs, ds, bs, cs, zs, ys;
  const float *A, *Dskip, *bias;
  void* y;
  const void* state;
  void* state_out;
  float* carry;  // a slot of a piece: ends [D, 4 NPL], sums of dt [D]
};

constexpr float kLog2e = 1.44269504f;

template <typename T>
__device__ __forceinline__ float as_float(T v) {
  if constexpr (std::is_same_v<T, uint16_t>) return __half2float(__ushort_as_half(v));
  else return __uint_as_float(v);
}

// max(v, 0) + log(1 + e), e = e^-|v|, by log(1 + e) = 2 atanh(s) = s P(s^2), s = e / (2 + e) <= 1/3: P of degree 4 is
// within 4.1e-9 (a fit at Chebyshev nodes). A NaN stays one: s is.
__device__ __forceinline__ float softplus(float v) {
  const float e = __builtin_amdgcn_exp2f(-fabsf(v) * kLog2e);
  const float s = e * __builtin_amdgcn_rcpf(2.0f + e), q = s * s;
  float p = fmaf(q, 0.2816145375705998f, 0.27964344707516564f);
  p = fmaf(p, q, 0.40024651333399913f);
  p = fmaf(p, q, 0.6666632040642534f);
  p = fmaf(p, q, 2.0000000077239766f);
  return fmaf(s, p, fmaxf(v, 0.0f));
}

__device__ __forceinline__ float silu(float v) {
  const float e = __builtin_amdgcn_exp2f(-fabsf(v) * kLog2e), r = __builtin_amdgcn_rcpf(1.0f + e);
  return v * (v < 0.0f ? e * r : r);
}

// a where mask is all ones, b where it is 0: a choice that stays one instruction, not a branch.
__device__ __forceinline__ float choose(uint32_t mask, float a, float b) {
  return __uint_as_float((__float_as_uint(a) & mask) | (__float_as_uint(b) & ~mask));
}

// A log2(e), finite: e^(0 A) is 1 for an infinite A too, as a row that does not count needs it.
__device__ __forceinline__ float decay_of(float a) { return __builtin_amdgcn_fmed3f(a * kLog2e, -3.402823466e38f, 3.402823466e38f) + 0.0f * (a != a ? a : 0.0f); }

// x of lane K of the four
template <int K>
__device__ __forceinline__ float lane4(float x) {
  return __builtin_bit_cast(float, __builtin_amdgcn_mov_dpp(__builtin_bit_cast(int, x), K * 0x55, 0xF, 0xF, true));
}

// p[s] is the lane's part of row s's sum; returns the four lanes' sum of row q = lane % 4.
__device__ __forceinline__ float join4(const float (&p)[4], int q) {
  const bool hi = q & 2, odd = q & 1;
  const float a = (hi ? p[2] : p[0]) + dpp_partner<2>(hi ? p[0] : p[2]);
  const float b = (hi ? p[3] : p[1]) + dpp_partner<2>(hi ? p[1] : p[3]);
  return (odd ? b : a) + dpp_partner<1>(odd ? a : b);
}

__device__ __forceinline__ float sum4(float v) {
  v += dpp_partner<1>(v);
  return v + dpp_partner<2>(v);
}

// A lane's states of one channel, in one load or store where the channel has 4 NPL.
template <int NPL>
__device__ __forceinline__ void load_state(const SscanParams& p, int64_t slot, bool has, int d, int q, float (&h)[NPL]) {
  const bool given = p.state && slot >= 0 && has;
  const int64_t at = (slot * p.D + d) * p.N + q * NPL;
#pragma unroll
  for (int j = 0; j < NPL; ++j) h[j] = 0.0f;
  if (!given) return;
  if (p.N == 4 * NPL) {
    if (p.sf16) {
      __half v[NPL];
      __builtin_memcpy(v, reinterpret_cast<const __half*>(p.state) + at, sizeof(v));
#pragma unroll
      for (int j = 0; j < NPL; ++j) h[j] = __half2float(v[j]);
    } else {
      __builtin_memcpy(h, reinterpret_cast<const float*>(p.state) + at, sizeof(h));
    }
    return;
  }
#pragma unroll
  for (int j = 0; j < NPL; ++j)
    if (q * NPL + j < p.N)
      h[j] = p.sf16 ? __half2float(reinterpret_cast<const __half*>(p.state)[at + j]) : reinterpret_cast<const float*>(p.state)[at + j];
}

template <int NPL>
__device__ __forceinline__ void store_state(const SscanParams& p, int64_t slot, int d, int q, const float (&h)[NPL]) {
  if (!p.state_out || slot < 0) return;
  const int64_t at = (slot * p.D + d) * p.N + q * NPL;
  if (p.N == 4 * NPL) {
    if (p.sf16) {
      __half v[NPL];
#pragma unroll
      for (int j = 0; j < NPL; ++j) v[j] = __float2half_rn(h[j]);
      __builtin_memcpy(reinterpret_cast<__half*>(p.state_out) + at, v, sizeof(v));
    } else {
      __builtin_memcpy(reinterpret_cast<float*>(p.state_out) + at, h, sizeof(h));
    }
    return;
  }
#pragma unroll
  for (int j = 0; j < NPL; ++j)
    if (q * NPL + j < p.N) {
      if (p.sf16) reinterpret_cast<__half*>(p.state_out)[at + j] = __float2half_rn(h[j]);
      else reinterpret_cast<float*>(p.state_out)[at + j] = h[j];
    }
}

template <int NPL>
__device__ __forceinline__ void load_decay(const SscanParams& p, int d, int q, float (&a)[NPL]) {
#pragma unroll
  for (int j = 0; j < NPL; ++j) a[j] = q * NPL + j < p.N ? decay_of(p.A[(int64_t)d * p.N + q * NPL + j]) : 0.0f;
}

constexpr int kRows = 32;  // rows of B and C in LDS at a time

constexpr int kBufferWord3 = 0x00020000;  // buffer resource word 3 for raw 32-bit access (gfx9)
constexpr uint32_t kNowhere = 0x80000000u;  // a byte offset behind every buffer below

// Rows t .. min(t + kRows, end) - 1 of a tensor (none of a null one). Loads past them give 0 and stores past them are
// dropped (the range check counts the scalar offset in), so no access needs a branch; strides of at most 2^23 elements
// keep kRows rows inside 32 bits.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t rows_rsrc(const void* p, int t, int end, int64_t stride, int size, int cols) {
  const int rows = p ? min(end - t, kRows) : 0;
  const char* q = reinterpret_cast<const char*>(p) + (rows > 0 ? t * stride * size : 0);
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<char*>(q), (short)0, rows > 0 ? (int)(((rows - 1) * stride + cols) * size) : 0, kBufferWord3);
}

template <typename T>
__device__ __forceinline__ T load1(__amdgpu_buffer_rsrc_t r, uint32_t voff, uint32_t soff) {
  if constexpr (sizeof(T) == 2) return (T)__builtin_amdgcn_raw_buffer_load_b16(r, voff, soff, 0);
  else return (T)__builtin_amdgcn_raw_buffer_load_b32(r, voff, soff, 0);
}

// f(0), ..., f(N - 1), as constants.
template <int N, typename F>
__device__ __forceinline__ void unrolled(F f) {
  if constexpr (N > 0) {
    unrolled<N - 1>(f);
    f(std::integral_constant<int, N - 1>());
  }
}

// u * b[J], of fp16 values in one instruction each.
template <int J>
__device__ __forceinline__ float times(float u, const uint32_t* b) { return u * __uint_as_float(b[J]); }
template <int J>
__device__ __forceinline__ float times(float u, const uint16_t* b) {
  uint32_t w;
  __builtin_memcpy(&w, b + (J & ~1), 4);
  float r;
  if constexpr (J & 1) asm("v_fma_mix_f32 %0, %1, %2, 0 op_sel:[0,1,0] op_sel_hi:[0,1,0]" : "=v"(r) : "v"(u), "v"(w));
  else asm("v_fma_mix_f32 %0, %1, %2, 0 op_sel_hi:[0,1,0]" : "=v"(r) : "v"(u), "v"(w));
  return r;
}

template <int NPL, typename T, typename Y>
struct Piece {
  static constexpr bool kY = !std::is_same_v<Y, void>;  // with y
  static constexpr int kNP = 4 * NPL, kBatches = kRows / 4, kPer = kRows * kNP / 256, kSize = sizeof(T);
  static constexpr int kYSize = std::is_same_v<Y, __half> ? 2 : 4;
  static constexpr int kAhead = kSize * NPL <= 8 ? 4 : kSize * NPL <= 16 ? 2 : 1;  // rows of B and C fetched ahead
  static constexpr int kAlign = kSize * NPL < 16 ? kSize * NPL : 16;
  const SscanParams& p;
  const int d, q, g;  // the lane's channel (clamped), its place in the four, the B/C group
  const bool live;
  T* const lds;       // [2][kRows][4][2][NPL]: a lane's values of B and C of a row side by side
  T xr[kBatches], dr[kBatches], zr[kBatches], br[kPer], cr[kPer];

  // x, delta and z of row t + 4 i + q, for batch i
  __device__ __forceinline__ void load_rows(int i, __amdgpu_buffer_rsrc_t rx, __amdgpu_buffer_rsrc_t rd, __amdgpu_buffer_rsrc_t rz) {
    const auto at = [&](__amdgpu_buffer_rsrc_t r, int64_t stride) {
      return load1<T>(r, (uint32_t)(q * (int)stride + d) * kSize, (uint32_t)(4 * i * (int)stride) * kSize);
    };
    xr[i] = at(rx, p.xs);
    dr[i] = at(rd, p.ds);
    if (kY) zr[i] = at(rz, p.zs);
  }

  // this thread's part of B and C: state k of rows row, row + 256 / kNP, ...
  __device__ __forceinline__ void load_bc(int t, int end) {
    const int k = threadIdx.x % kNP, row = threadIdx.x / kNP, cols = p.G * p.N;
    const auto rb = rows_rsrc(p.B, t, end, p.bs, kSize, cols), rc = rows_rsrc(kY ? p.C : nullptr, t, end, p.cs, kSize, cols);
    const uint32_t vb = k < p.N ? (uint32_t)(row * (int)p.bs + g * p.N + k) * kSize : kNowhere;
    const uint32_t vc = k < p.N ? (uint32_t)(row * (int)p.cs + g * p.N + k) * kSize : kNowhere;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      br[i] = load1<T>(rb, vb, (uint32_t)(i * (256 / kNP) * (int)p.bs) * kSize);
      if (kY) cr[i] = load1<T>(rc, vc, (uint32_t)(i * (256 / kNP) * (int)p.cs) * kSize);
    }
  }

  __device__ __forceinline__ void store_bc(int buf) {
    const int k = threadIdx.x % kNP, row = threadIdx.x / kNP;
    T* at = lds + ((buf * kRows + row) * 4 + k / NPL) * 2 * NPL + k % NPL;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      at[i * (256 / kNP) * 2 * kNP] = br[i];
      if (kY) at[i * (256 / kNP) * 2 * kNP + NPL] = cr[i];
    }
  }

  // Rows begin .. end - 1 from the state in h, which becomes the state behind them; returns the sum of dt (the
  // lane's rows; without y only).
  __device__ __forceinline__ float run(int begin, int end, const float (&a)[NPL], float (&h)[NPL]) {
    const float bias = p.bias ? p.bias[d] : 0.0f, skip = kY && p.Dskip ? p.Dskip[d] : 0.0f;
    const uint32_t sp = p.softplus ? ~0u : 0u, gate = p.z ? ~0u : 0u;
    const uint32_t yv = live ? (uint32_t)(q * (int)p.ys + d) * kYSize : kNowhere, ystep = (uint32_t)(4 * (int)p.ys) * kYSize;
    float sum = 0.0f;
    const auto rx_of = [&](int t) { return rows_rsrc(p.x, t, end, p.xs, kSize, p.D); };
    const auto rd_of = [&](int t) { return rows_rsrc(p.delta, t, end, p.ds, kSize, p.D); };
    const auto rz_of = [&](int t) { return rows_rsrc(kY ? p.z : nullptr, t, end, p.zs, kSize, p.D); };
    load_bc(begin, end);
    {
      const auto rx = rx_of(begin), rd = rd_of(begin), rz = rz_of(begin);
#pragma unroll
      for (int i = 0; i < kBatches; ++i) load_rows(i, rx, rd, rz);
    }
    store_bc(0);
    __syncthreads();
    int buf = 0;
    for (int t = begin; t < end; t += kRows, buf ^= 1) {
      // (behind the last rows these are empty)
      const auto rx = rx_of(t + kRows), rd = rd_of(t + kRows), rz = rz_of(t + kRows);
      const auto ry = rows_rsrc(kY ? p.y : nullptr, t, end, p.ys, kYSize, p.D);
      load_bc(t + kRows, end);
      const T* rows = lds + buf * kRows * 2 * kNP + q * 2 * NPL;
      T now[kAhead][2 * NPL], next[kAhead][2 * NPL];
      const auto fetch = [&](int unit) {
#pragma unroll
        for (int n = 0; n < kAhead; ++n)
          __builtin_memcpy(next[n], __builtin_assume_aligned(rows + (unit * kAhead + n) * 2 * kNP, kAlign), (kY ? 2 : 1) * sizeof(T) * NPL);
      };
      fetch(0);
#pragma unroll
      for (int i = 0; i < kBatches; ++i) {
        if (i % 2 == 0 && t + 4 * i >= end) break;
        const float x = as_float(xr[i]), dl = as_float(dr[i]) + bias, z = kY ? as_float(zr[i]) : 0.0f;
        load_rows(i, rx, rd, rz);  // the next rows' into their place
        // past the end: dt 0, and u too (x is 0 there)
        const float dt = q < end - t - 4 * i ? choose(sp, softplus(dl), dl) : 0.0f, u = dt * x;
        if (!kY) sum += dt;
        float part[4];
        const auto step = [&](auto k) {
          constexpr int K = decltype(k)::value;
          const int unit = (4 * i + K) / kAhead;
          if (K % kAhead == 0) {
#pragma unroll
            for (int n = 0; n < kAhead; ++n) {
#pragma unroll
              for (int j = 0; j < 2 * NPL; ++j) now[n][j] = next[n][j];
            }
            // the next rows' values are on their way while these are used (and no further ones: they would fill the registers)
            if (unit + 1 < kRows / kAhead) fetch(unit + 1);
            asm volatile("" ::: "memory");
          }
          const float ds = lane4<K>(dt), us = lane4<K>(u);
          const T* bq = now[K % kAhead];
          part[K] = 0.0f;
          unrolled<NPL>([&](auto n) {
            constexpr int j = decltype(n)::value;
            h[j] = fmaf(__builtin_amdgcn_exp2f(ds * a[j]), h[j], times<j>(us, bq));
            if (kY) part[K] = fmaf(as_float(bq[NPL + j]), h[j], part[K]);
          });
        };
        unrolled<4>(step);
        if constexpr (kY) {
          const float y = fmaf(skip, x, join4(part, q)) * choose(gate, silu(z), 1.0f);
          if constexpr (kYSize == 2) __builtin_amdgcn_raw_buffer_store_b16(__half_as_ushort(__float2half_rn(y)), ry, yv, i * ystep, 0);
          else __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(y), ry, yv, i * ystep, 0);
        }
      }
      if (end - t > kRows) {
        store_bc(buf ^ 1);
        __syncthreads();
      }
    }
    return sum;
  }
};

// The state that enters piece `chunk` where steps below zero make a piece's decay grow out of fp32's range: it is taken as a
// value of at most 1 and a power of two, so that a state of 0, or one small enough, goes through as row by row. Rare, so it
// is a pass of its own behind the ordinary one.
template <int NPL>
__device__ __forceinline__ void fold_growing(const float (&a)[NPL], const float* from, const float* sums, int64_t size, int chunk, float (&h)[NPL]) {
#pragma unroll
  for (int j = 0; j < NPL; ++j) h[j] = from[j];
  for (int c = 1; c < chunk; ++c) {
    const float s = sums[c * size];
#pragma unroll
    for (int j = 0; j < NPL; ++j) {
      // (2^1000 takes every state but 0 out of range; a NaN has made the piece's end one)
      const float x = __builtin_amdgcn_fmed3f(s * a[j], -1000.0f, 1000.0f), n = ceilf(x);
      h[j] = __builtin_ldexpf(h[j] * __builtin_amdgcn_exp2f(x - n), (int)n) + from[c * size + j];
    }
  }
}

// ENDS: the ends of the pieces that have one behind them, the first ones' from the initial state (with their y unless
// Y is void), the others' from zero. Else every other piece with y, from the state that it folds from the ends.
template <int NPL, typename T, typename Y, bool ENDS>
__global__ __launch_bounds__(256) void k_selective_scan(SscanParams p) {
  constexpr int kNP = 4 * NPL;
  __shared__ __align__(16) T lds[2 * kRows * 2 * kNP];
  const int blocks = p.G * p.per_group, cb = blockIdx.x % blocks;
  const int64_t at = blockIdx.x / blocks;  // piece: sequence i has begin(i) / piece + i and the ones behind it
  const Seqs& sq = p.seq;
  int i;
  if (sq.offsets) i = last_not_above(sq.nseq, at, [&](int k) { return (int64_t)(seq_begin(sq, k) / p.piece + k); });
  else i = last_not_above(sq.nseq, at, [&](int k) { return (int64_t)(k * sq.each / p.piece + k); });
  const int begin = uniform(seq_begin(sq, i)), end = uniform(seq_end(sq, i, begin));
  const int chunk = (int)(at - (begin / p.piece + i)), pieces = max((int)(((uint32_t)(end - begin) + p.piece - 1) / (uint32_t)p.piece), 1);
  if (chunk < 0 || chunk >= pieces) return;
  const bool last = chunk == pieces - 1;
  if (ENDS ? last : p.first && chunk == 0 && !last) return;
  const int g = cb / p.per_group, q = threadIdx.x & 3;
  const int dg = cb % p.per_group * 64 + (threadIdx.x >> 2);
  const int d = g * p.Dg + min(dg, p.Dg - 1);
  const bool live = dg < p.Dg;
  float a[NPL], h[NPL];
  load_decay(p, d, q, a);
  const int64_t slot = seq_slot(sq, i);
  const int64_t size = (int64_t)p.D * (kNP + 1);
  const int64_t carry = qssm_sscan::first_slot(i, begin / p.piece) + chunk;  // (a sequence of one piece has none)
  float* ends = p.carry + carry * size + (int64_t)d * kNP + q * NPL;
#pragma unroll
  for (int j = 0; j < NPL; ++j) h[j] = 0.0f;
  if (chunk == 0 && (last || ENDS)) {
    load_state(p, slot, !sq.has || sq.has[i] != 0, d, q, h);
    // the last piece's slot has no ends: it keeps the initial state, which the last piece may overwrite in `state`
    if (std::is_same_v<Y, void> && live) {
#pragma unroll
      for (int j = 0; j < NPL; ++j) ends[(pieces - 1) * size + j] = h[j];
    }
  } else if (!ENDS && chunk == 0) {
#pragma unroll
    for (int j = 0; j < NPL; ++j) h[j] = ends[(pieces - 1) * size + j];
  } else if (!ENDS) {
    const float* from = ends - chunk * size;
    const float* sums = p.carry + (carry - chunk) * size + (int64_t)p.D * kNP + d;
    float most = 0.0f;
#pragma unroll
    for (int j = 0; j < NPL; ++j) h[j] = from[j];
#pragma unroll 4
    for (int c = 1; c < chunk; ++c) {
      const float s = sums[c * size];
#pragma unroll
      for (int j = 0; j < NPL; ++j) {
        const float x = s * a[j];
        most = fmaxf(most, x);
        h[j] = fmaf(__builtin_amdgcn_exp2f(x), h[j], from[c * size + j]);
      }
    }
    if (most > 126.0f) fold_growing<NPL>(a, from, sums, size, chunk, h);
  }
  const int b = begin + chunk * p.piece, e = last ? end : b + p.piece;
  if (ENDS && (chunk > 0 || std::is_same_v<Y, void>)) {
    const float sum = sum4(Piece<NPL, T, void>{p, d, q, g, live, lds}.run(b, e, a, h));
    if (live && q == 0) p.carry[carry * size + (int64_t)p.D * kNP + d] = sum;
  } else if (b < e) {
    Piece<NPL, T, Y>{p, d, q, g, live, lds}.run(b, e, a, h);
  }
  if (!live) return;
  if (last) {
    store_state(p, slot, d, q, h);
  } else if (ENDS) {
#pragma unroll
    for (int j = 0; j < NPL; ++j) ends[j] = h[j];
  }
}

// One row a sequence: four lanes own a channel of one sequence (R = 1) or of four (R = 4), where each lane prepares one
// sequence's dt, x and gate for all four, as a batch of the scan does. The bytes of the states bound it, but a wave's many
// small loads cost as much: 256 sequences, 4096 channels, 16 fp32 states take 44 us with R = 1, and 35 with R = 4.
template <int NPL, int R, typename T>
__global__ __launch_bounds__(256) void k_selective_step(SscanParams p) {
  const int cb = blockIdx.x % (p.G * p.per_group), g = cb / p.per_group, q = threadIdx.x & 3;
  const int dg = cb % p.per_group * 64 + (threadIdx.x >> 2);
  const int d = g * p.Dg + min(dg, p.Dg - 1);
  const int i0 = (int)(blockIdx.x / (p.G * p.per_group)) * R, mine = R == 4 ? i0 + q : i0;
  const bool live = dg < p.Dg && mine < p.seq.nseq;
  float h[R][NPL];
  T b[R][NPL], c[R][NPL];
  int64_t slot[R];
  const auto part = [&](const void* from, int64_t at, T (&to)[NPL]) {
    const T* v = reinterpret_cast<const T*>(from) + at + g * p.N + q * NPL;
    if (p.N == 4 * NPL) {
      __builtin_memcpy(to, v, sizeof(to));
    } else {
#pragma unroll
      for (int j = 0; j < NPL; ++j) to[j] = q * NPL + j < p.N ? v[j] : T(0);
    }
  };
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const int i = min(i0 + r, p.seq.nseq - 1);
    slot[r] = seq_slot(p.seq, i);
    load_state(p, slot[r], !p.seq.has || p.seq.has[i] != 0, d, q, h[r]);
    part(p.B, (int64_t)i * p.bs, b[r]);
    part(p.C, (int64_t)i * p.cs, c[r]);
  }
  const int64_t i = min(mine, p.seq.nseq - 1);
  const float x = as_float(reinterpret_cast<const T*>(p.x)[i * p.xs + d]);
  const float v = as_float(reinterpret_cast<const T*>(p.delta)[i * p.ds + d]) + (p.bias ? p.bias[d] : 0.0f);
  const float z = p.z ? as_float(reinterpret_cast<const T*>(p.z)[i * p.zs + d]) : 0.0f;
  const float skip = p.Dskip ? p.Dskip[d] : 0.0f;
  float a[NPL];
  load_decay(p, d, q, a);
  const float dt = p.softplus ? softplus(v) : v, u = dt * x;
  float sum[4];
  unrolled<R>([&](auto k) {
    constexpr int K = decltype(k)::value;
    const float ds = R == 4 ? lane4<K>(dt) : dt, us = R == 4 ? lane4<K>(u) : u;
    sum[K] = 0.0f;
#pragma unroll
    for (int j = 0; j < NPL; ++j) {
      h[K][j] = fmaf(__builtin_amdgcn_exp2f(ds * a[j]), h[K][j], us * as_float(b[K][j]));
      sum[K] = fmaf(as_float(c[K][j]), h[K][j], sum[K]);
    }
    if (dg < p.Dg && i0 + K < p.seq.nseq) store_state(p, slot[K], d, q, h[K]);
  });
  float y;
  if constexpr (R == 4) y = join4(sum, q);
  else y = sum4(sum[0]);
  y = fmaf(skip, x, y);
  if (p.z) y *= silu(z);
  if (live && (R == 4 || q == 0)) {
    if (p.yf16) reinterpret_cast<__half*>(p.y)[i * p.ys + d] = __float2half_rn(y);
    else reinterpret_cast<float*>(p.y)[i * p.ys + d] = y;
  }
}

constexpr int64_t kMaxBlocks = ((int64_t)1 << 24) - 1;  // a grid holds fewer than 2^32 threads

int npl_of(int64_t N) { return N <= 8 ? 2 : N <= 16 ? 4 : N <= 32 ? 8 : 16; }

int64_t blocks_of(const qssm_sscan_args& a) { return a.ngroups * cdiv(a.dim / a.ngroups, 64); }

int64_t piece_rows(const qssm_sscan_args& a) { return qssm_sscan::piece_rows(a.tokens, a.nseq, 4 * blocks_of(a), a.seq_offsets); }

bool is_cut(const qssm_sscan_args& a, int64_t piece) { return qssm_sscan::is_cut(a.tokens, a.nseq, piece, a.seq_offsets); }

size_t slot_bytes(int64_t dim, int64_t dstate) { return (size_t)dim * (size_t)(4 * npl_of(dstate) + 1) * sizeof(float); }

size_t carry_bytes(const qssm_sscan_args& a, int64_t piece) {
  return (size_t)qssm_sscan::carry_slots(a.tokens, a.nseq, piece) * slot_bytes(a.dim, a.dstate);
}

// First pieces in full with the others' ends: a pass less of their rows, but the first launch then waits for rows with y.
// It gains where the second one has sequences of different lengths to level out (16384 rows, 4096 channels in 24
// of them: 458 us without, 435 with; in 100, 1536 channels: 221, 199; 8192 rows, 2048 channels in 4: 144, 141), and costs
// where it does not (8 of 1024 rows, 1536 channels: 103, 109; one of 8192: 121, 124).
bool runs_first(const qssm_sscan_args& a) { return a.seq_offsets && a.nseq > 1; }

bool is_step(const qssm_sscan_args& a) { return !a.seq_offsets && a.tokens == a.nseq; }

template <int NPL, typename T, typename Y>
qssm_status launch_scan(const SscanParams& p, const qssm_sscan_args& a, int64_t blocks, hipStream_t stream) {
  if (is_cut(a, p.piece)) {
    if (p.first) k_selective_scan<NPL, T, Y, true><<<(unsigned)blocks, 256, 0, stream>>>(p);
    else k_selective_scan<NPL, T, void, true><<<(unsigned)blocks, 256, 0, stream>>>(p);
    if (const qssm_status s = launch_status("selective_scan")) return s;
  }
  k_selective_scan<NPL, T, Y, false><<<(unsigned)blocks, 256, 0, stream>>>(p);
  return launch_status("selective_scan");
}

template <int NPL, typename T>
qssm_status launch(SscanParams p, const qssm_sscan_args& a, hipStream_t stream) {
  if (is_step(a)) {
    const bool four = qssm_sscan::four_at_a_time(a.nseq, blocks_of(a), NPL);
    const int64_t blocks = (four ? cdiv(a.nseq, 4) : a.nseq) * blocks_of(a);
    if (blocks > kMaxBlocks) return fail(QSSM_ERR_UNSUPPORTED, "nseq * dim above 2^30");
    if (four) k_selective_step<NPL, NPL <= 8 ? 4 : 1, T><<<(unsigned)blocks, 256, 0, stream>>>(p);
    else k_selective_step<NPL, 1, T><<<(unsigned)blocks, 256, 0, stream>>>(p);
    return launch_status("selective_scan");
  }
  const int64_t blocks = (a.tokens / p.piece + a.nseq) * blocks_of(a);
  if (blocks > kMaxBlocks) return fail(QSSM_ERR_UNSUPPORTED, "tokens * dim too large");
  return p.yf16 ? launch_scan<NPL, T, __half>(p, a, blocks, stream) : launch_scan<NPL, T, float>(p, a, blocks, stream);
}

template <typename T>
qssm_status launch_n(const SscanParams& p, const qssm_sscan_args& a, hipStream_t stream) {
  switch (npl_of(a.dstate)) {
    case 2: return launch<2, T>(p, a, stream);
    case 4: return launch<4, T>(p, a, stream);
    case 8: return launch<8, T>(p, a, stream);
    default: return launch<16, T>(p, a, stream);
  }
}

// The sizes alone: what the workspace depends on.
qssm_status check_sizes(const qssm_sscan_args& a) {
  if (const qssm_status s = check_seqs(a.tokens, a.dim, a.nseq, a.seq_offsets, a.state, a.state_out, a.slots, a.state_slots)) return s;
  if (a.dstate < 1 || a.dstate > 64) return fail(QSSM_ERR_UNSUPPORTED, "dstate must be in 1..64");
  if (a.ngroups < 1 || a.dim % a.ngroups != 0) return fail(QSSM_ERR_INVALID_ARG, "dim is not a multiple of ngroups");
  return QSSM_OK;
}

}  // namespace

extern "C" size_t qssm_selective_scan_workspace_size(const qssm_sscan_args* a) {
  clear_error();
  if (!a || check_sizes(*a) != QSSM_OK || a->nseq == 0 || a->dim == 0 || is_step(*a)) return 0;
  const int64_t piece = piece_rows(*a);
  return is_cut(*a, piece) ? carry_bytes(*a, piece) : 0;
}

extern "C" size_t qssm_selective_scan_workspace_bound(int64_t tokens, int64_t dim, int64_t dstate, int32_t ngroups) {
  qssm_sscan_args a{};
  a.tokens = tokens, a.dim = dim, a.dstate = dstate, a.ngroups = ngroups, a.nseq = 1;
  clear_error();
  if (check_sizes(a) != QSSM_OK || dim == 0) return 0;
  return (size_t)qssm_sscan::most_slots(tokens, 4 * blocks_of(a)) * slot_bytes(dim, dstate);
}

extern "C" qssm_status qssm_selective_scan(const qssm_sscan_args* a, void* workspace, size_t workspace_bytes,
                                           hipStream_t stream) {
  clear_error();
  if (!a) return fail(QSSM_ERR_INVALID_ARG, "args is null");
  if (const qssm_status s = check_sizes(*a)) return s;
  const int64_t T = a->tokens, D = a->dim, N = a->dstate, GN = a->ngroups * N;
  if (a->io_dtype != QSSM_F32 && a->io_dtype != QSSM_F16) return fail(QSSM_ERR_INVALID_ARG, "io_dtype must be QSSM_F32 or QSSM_F16");
  if (a->y_dtype != QSSM_F32 && a->y_dtype != QSSM_F16) return fail(QSSM_ERR_INVALID_ARG, "y_dtype must be QSSM_F32 or QSSM_F16");
  if (a->state_dtype != QSSM_F32 && a->state_dtype != QSSM_F16)
    return fail(QSSM_ERR_INVALID_ARG, "state_dtype must be QSSM_F32 or QSSM_F16");
  if (a->reserved != 0) return fail(QSSM_ERR_INVALID_ARG, "reserved must be 0");
  for (const int64_t stride : {a->x_stride, a->delta_stride, a->B_stride, a->C_stride, a->z_stride, a->y_stride})
    if (stride > (1 << 23)) return fail(QSSM_ERR_UNSUPPORTED, "a stride above 2^23");
  const int64_t sx = type_size(a->io_dtype), sy = type_size(a->y_dtype), ss = type_size(a->state_dtype);
  if (const qssm_status s = check_rows("x", a->x, T, D, a->x_stride, sx)) return s;
  if (const qssm_status s = check_rows("delta", a->delta, T, D, a->delta_stride, sx)) return s;
  if (const qssm_status s = check_rows("B", a->B, T, GN, a->B_stride, sx)) return s;
  if (const qssm_status s = check_rows("C", a->C, T, GN, a->C_stride, sx)) return s;
  if (const qssm_status s = check_rows("z", a->z, T, D, a->z_stride, sx)) return s;
  if (const qssm_status s = check_rows("y", a->y, T, D, a->y_stride, sy)) return s;
  if (a->nseq == 0 || D == 0) return QSSM_OK;
  if (!a->A || (T > 0 && (!a->x || !a->delta || !a->B || !a->C || !a->y)))
    return fail(QSSM_ERR_INVALID_ARG, "null required pointer");
  if (((uintptr_t)a->A | (uintptr_t)a->Dskip | (uintptr_t)a->delta_bias) % 4 != 0 ||
      ((uintptr_t)a->state | (uintptr_t)a->state_out) % ss != 0)
    return fail(QSSM_ERR_INVALID_ARG, "A, Dskip, delta_bias or a state is not aligned to its type");
  if (a->slots > ((int64_t)1 << 58) / (D * N)) return fail(QSSM_ERR_UNSUPPORTED, "slots * dim * dstate above 2^58");
  SscanParams p{};
  p.piece = (int32_t)piece_rows(*a);
  p.first = runs_first(*a);
  const size_t need = !is_step(*a) && is_cut(*a, p.piece) ? carry_bytes(*a, p.piece) : 0;
  if (need && (!workspace || workspace_bytes < need))
    return fail(QSSM_ERR_WORKSPACE, "workspace of %zu bytes, %zu needed", workspace ? workspace_bytes : (size_t)0, need);
  if (need && (uintptr_t)workspace % 16 != 0) return fail(QSSM_ERR_INVALID_ARG, "workspace is not 16-byte aligned");
  const int64_t sb = a->slots * D * N * ss;
  const Span y{a->y, T, a->y_stride * sy, D * sy}, out = flat(a->state_out, sb), ws = flat(need ? workspace : nullptr, (int64_t)need);
  const Span in[] = {{a->x, T, a->x_stride * sx, D * sx},       {a->delta, T, a->delta_stride * sx, D * sx},
                     {a->B, T, a->B_stride * sx, GN * sx},      {a->C, T, a->C_stride * sx, GN * sx},
                     {a->z, T, a->z_stride * sx, D * sx},       flat(a->A, D * N * 4),
                     flat(a->Dskip, D * 4),                     flat(a->delta_bias, D * 4),
                     flat(a->seq_offsets, (a->nseq + 1) * 4),   flat(a->state_slots, a->nseq * 4),
                     flat(a->has_state, a->nseq)};
  for (const Span& s : in)
    if (overlap(y, s) || overlap(out, s) || overlap(ws, s))
      return fail(QSSM_ERR_INVALID_ARG, "y, state_out or the workspace overlaps an input");
  const Span st = flat(a->state, sb);
  if (overlap(y, st) || overlap(y, out) || overlap(y, ws) || overlap(ws, st) || overlap(ws, out) ||
      (a->state_out != a->state && overlap(out, st)))
    return fail(QSSM_ERR_INVALID_ARG, "y, state, state_out and the workspace overlap");
  p.seq = make_seqs(T, a->nseq, a->seq_offsets, a->state_slots, a->has_state, a->slots);
  p.D = (int32_t)D;
  p.N = (int32_t)N;
  p.G = a->ngroups;
  p.Dg = (int32_t)(D / a->ngroups);
  p.per_group = (int32_t)cdiv(p.Dg, 64);
  p.softplus = a->delta_softplus != 0;
  p.yf16 = a->y_dtype == QSSM_F16;
  p.sf16 = a->state_dtype == QSSM_F16;
  p.x = a->x, p.xs = a->x_stride;
  p.delta = a->delta, p.ds = a->delta_stride;
  p.B = a->B, p.bs = a->B_stride;
  p.C = a->C, p.cs = a->C_stride;
  p.z = a->z, p.zs = a->z_stride;
  p.y = a->y, p.ys = a->y_stride;
  p.A = a->A, p.Dskip = a->Dskip, p.bias = a->delta_bias;
  p.state = a->state, p.state_out = a->state_out;
  p.carry = static_cast<float*>(workspace);
  return a->io_dtype == QSSM_F16 ? launch_n<uint16_t>(p, *a, stream) : launch_n<uint32_t>(p, *a, stream);
}
