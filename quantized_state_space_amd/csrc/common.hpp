// Shared device helpers and host-side error handling of libqssm (gfx950 only).
#pragma once

#include <hip/hip_runtime.h>
#include <hip/hip_fp16.h>
#include <stdint.h>

#include <algorithm>
#include <numeric>

#include "qssm.h"

namespace qssm {

// ---------------------------------------------------------------------------------------------
// Host: error reporting (thread-local message, never an exception across the ABI).
qssm_status fail(qssm_status code, const char* fmt, ...) __attribute__((format(printf, 2, 3)));
void clear_error();
// Maps a pending launch error to QSSM_ERR_DEVICE (with the runtime's message).
qssm_status launch_status(const char* what);

// Ceil division for launch geometry.
inline int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Where a tensor lies: `rows` rows of `width` bytes, `stride` bytes apart (at least the width).
struct Span {
  const void* p;
  int64_t rows, stride, width;
};

inline Span flat(const void* p, int64_t bytes) { return Span{p, 1, bytes, bytes}; }

// Whether a row of a shares a byte with a row of b (a tensor that is null or empty shares none). Exact where the
// strides are equal or a tensor has one row. Tensors of two strides whose ranges meet are apart if their rows
// are modulo the strides' greatest common divisor (columns of wider tensors), and taken to overlap otherwise.
inline bool overlap(Span a, Span b) {
  if (!a.p || !b.p || a.rows * a.width == 0 || b.rows * b.width == 0) return false;
  const int64_t d = (int64_t)((uintptr_t)b.p - (uintptr_t)a.p);
  if (d >= (a.rows - 1) * a.stride + a.width || -d >= (b.rows - 1) * b.stride + b.width) return false;
  if (a.rows == 1) a.stride = b.stride;
  if (b.rows == 1) b.stride = a.stride;
  if (a.stride == b.stride) {
    // row j of b and row i of a meet where -b.width < d + (j - i) stride < a.width: the least such j - i
    const int64_t s = a.stride, low = -b.width - d;
    const int64_t k = std::max((low >= 0 ? low / s : -((s - 1 - low) / s)) + 1, 1 - a.rows);
    return k <= b.rows - 1 && d + k * s < a.width;
  }
  const int64_t g = std::gcd(a.stride, b.stride), m = (d % g + g) % g;
  return m < a.width || m + b.width > g;
}

// ---------------------------------------------------------------------------------------------
// Device: the quantization rule.
//
// q = clamp(RNE(v / s), lo, hi) with v / s the exact rational quotient (Quamba2's 8-bit codes,
// rounding half to even, saturating). The fp32 division is correctly rounded, and rounding is
// monotone, so rint() of the fp32 quotient f differs from the exact RNE only when f itself is a
// half-integer k + 1/2 while the exact quotient is not: then the sign of the exact remainder
// v - f*s, which one fused multiply-add yields without intermediate rounding, decides the side.
// Valid scales lie in [2^-100, 2^100]; there every non-zero remainder is at least 2^-149 in
// magnitude, so its sign survives the final rounding of the fma.
__host__ __device__ __forceinline__ bool scale_ok(float s) { return s >= 0x1p-100f && s <= 0x1p100f; }

__host__ __device__ __forceinline__ int rne_sat(float v, float s, float lo, float hi) {
  float f = v / s;
  float r = rintf(f);
  if (fabsf(f - r) == 0.5f) {
    float rem = fmaf(-f, s, v);
    if (rem > 0.0f) r = f + 0.5f;
    else if (rem < 0.0f) r = f - 0.5f;
  }
  r = fminf(fmaxf(r, lo), hi);
  return (v != v) ? 0 : (int)r;  // NaN encodes as 0
}

__host__ __device__ __forceinline__ int8_t quant8(float v, float s) {
  return scale_ok(s) ? (int8_t)rne_sat(v, s, -128.0f, 127.0f) : (int8_t)0;
}

// The same rule from a reciprocal r = fl32(1/s), for which |v*r - v/s| <= 2^-23 |v/s| + 2^-48 |v/s|
// <= 3.1e-5 when |v/s| <= 256. Let f = v*r clamped to [-256, 256] (beyond that the code saturates
// anyway) and c = rint(f). If |f - c| <= 1/2 - 2^-14, the exact quotient d lies within
// 1/2 - 2^-14 + 3.1e-5 < 1/2 of c and RNE(d) = c. Otherwise d may sit on or beyond the
// half-integer b = c +- 1/2 on f's side of c (d is within 1/2 of f). The exact v - b*s is a multiple of 2^-149 (b is a multiple of 1/2 and s >= 2^-102 in
// every use), so the single rounding of fmaf(-b, s, v) keeps its sign and its zero-ness:
// beyond b moves to the neighbour c +- 1, exactly on b is a tie resolved to the even neighbour.
// The rare near-boundary branch is skipped by a whole wave when none of its lanes needs it.
// Returns the unsaturated code as a float; the caller clamps and handles NaN and invalid scales.
__host__ __device__ __forceinline__ float rne_recip(float v, float s, float r) {
  const float f = fminf(fmaxf(v * r, -256.0f), 256.0f);
  float c = rintf(f);
  const float t = f - c;
  if (fabsf(t) > 0.5f - 0x1p-14f) {
    const float h = copysignf(0.5f, t);
    const float e = fmaf(-(c + h), s, v);
    const float eh = (h > 0.0f) ? e : -e;        // > 0: beyond the boundary on f's side
    const bool odd = (c * 0.5f) != rintf(c * 0.5f);
    if (eh > 0.0f || (eh == 0.0f && odd)) c += h + h;
  }
  return c;
}

__host__ __device__ __forceinline__ int rne_sat_recip(float v, float s, float r, int lo, int hi) {
  const float c = fminf(fmaxf(rne_recip(v, s, r), (float)lo), (float)hi);
  return (v == v) ? (int)c : 0;  // NaN encodes as 0
}

// Reciprocal used with rne_sat_recip; 0 marks a scale outside the valid range (codes 0).
__host__ __device__ __forceinline__ float recip_or_zero(float s) { return scale_ok(s) ? 1.0f / s : 0.0f; }

__host__ __device__ __forceinline__ int8_t quant8_r(float v, float s, float r) {
  return (r != 0.0f) ? (int8_t)rne_sat_recip(v, s, r, -128, 127) : (int8_t)0;
}

// Soft-edge byte (Quamba-SE blog, 2.1 and 2.2): strict |v| < L selects scale/m with a 6-bit
// payload (tag 10), |v| > H selects scale*m (tag 11), anything else (including both tests true)
// the base scale with a 7-bit payload (tag 0). Payloads are two's complement. The mode ratio m is 4
// (sections 2.1-2.2) or 2 (the shift-only form of section 4.1); im = 1/m. r = recip_or_zero(s):
// the small and large modes scale s and r by exact powers of two.
__host__ __device__ __forceinline__ uint8_t softedge_code_r(float v, float s, float r, float L, float H,
                                                            float m, float im) {
  if (r == 0.0f) return 0;
  const float a = fabsf(v);
  const bool small = a < L, large = a > H;
  const bool sm = small && !large, lg = large && !small;
  const float ss = sm ? im * s : (lg ? m * s : s);
  const float rr = sm ? m * r : (lg ? im * r : r);
  const int lim = (sm || lg) ? 32 : 64;
  const int q = rne_sat_recip(v, ss, rr, -lim, lim - 1);
  const uint32_t code = sm ? (0x80u | ((uint32_t)q & 0x3Fu))
                           : (lg ? (0xC0u | ((uint32_t)q & 0x3Fu)) : ((uint32_t)q & 0x7Fu));
  return (uint8_t)code;  // NaN: neither small nor large, payload 0
}

// Value of a soft-edge byte in units of the base scale: the payload times 1, 1/m or m (exact).
__host__ __device__ __forceinline__ float softedge_unit(uint32_t b, float m, float im) {
  if ((b & 0x80u) == 0) return (float)((b & 0x40u) ? (int)(b & 0x7Fu) - 128 : (int)(b & 0x7Fu));
  const int q = (b & 0x20u) ? (int)(b & 0x3Fu) - 64 : (int)(b & 0x3Fu);
  return (float)q * ((b & 0x40u) ? m : im);
}

// Value of a soft-edge byte as one correctly rounded fp32 product (0 for an invalid scale):
// the exact unit times s (m * s and im * s are exact for a valid s, so unit * s rounds once).
__host__ __device__ __forceinline__ float softedge_value(uint32_t b, float s, float m, float im) {
  if (!scale_ok(s)) return 0.0f;
  if ((b & 0x80u) == 0) return softedge_unit(b, m, im) * s;
  const int q = (b & 0x20u) ? (int)(b & 0x3Fu) - 64 : (int)(b & 0x3Fu);
  return (float)q * ((b & 0x40u) ? s * m : s * im);
}

// Mode ratio of a soft-edge code type (QSSM_X_SOFTEDGE: 4, QSSM_X_SOFTEDGE2: 2).
__host__ __device__ __forceinline__ float softedge_ratio(int code_type) {
  return code_type == QSSM_X_SOFTEDGE2 ? 2.0f : 4.0f;
}

// Scale from a group absmax (device side of compute_scales): fl32(absmax / 127), 0 -> 1,
// clamped to the valid range.
__device__ __forceinline__ float scale_from_absmax(float a) {
  if (a == 0.0f) return 1.0f;
  float s = a / 127.0f;
  return fminf(fmaxf(s, 0x1p-100f), 0x1p100f);
}

// Scale of one row from its absmax, where a kernel makes a scale for every row: the product with
// fl32(1/127) (within one unit in the last place of absmax / 127, without a division), 0 -> 1, clamped
// to the valid range. absmax / scale stays below 127.0001.
__device__ __forceinline__ float row_scale(float a) {
  if (a == 0.0f) return 1.0f;
  return fminf(fmaxf(a * (1.0f / 127.0f), 0x1p-100f), 0x1p100f);
}

// |v| if finite, else 0 (absmax ignores NaN and infinities).
__device__ __forceinline__ float finite_abs(float v) {
  float a = fabsf(v);
  return (a <= 3.402823466e38f) ? a : 0.0f;
}

// Codes of N values with one scale, packed little-endian: clamp(RNE(v / s), -128, 127), NaN 0, every
// code 0 for an invalid scale (the rule above). With r ~ 1/s, adding 1.5 * 2^23 in the fused
// multiply-add leaves c = RNE(v r) in the low bits of m. c is the nearest code when the remainder
// e = v - c s is inside (-s/2, s/2): the fma rounds it once, rounding is monotone and s/2 is a
// float, so |e| < s/2 after rounding implies it before. That fails only within ~2^-16 of a
// half-integer (or for a NaN); a lane with such a value decides all its codes by quant8_r. Values are
// clamped to [-128 s, 127 s] first (fl(127 s) / s still rounds to 127). IN_RANGE: the caller knows
// that every value is finite and |v| <= 127.4 s, as with the scale of the row's own absmax.
template <bool IN_RANGE, int N>
__device__ __forceinline__ void quant_row(const float (&v)[N], float s, uint32_t (&w)[N / 4]) {
  constexpr float kMagic = 12582912.0f;
  const bool ok = scale_ok(s);
  const float r = __builtin_amdgcn_rcpf(s);  // 1 ulp: the remainder decides, not r
  const float half = 0.5f * s, hi = 127.0f * s, lo = -128.0f * s;
  uint32_t m[N];
  bool bad = !ok;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const float x = IN_RANGE ? v[i] : __builtin_amdgcn_fmed3f(v[i], lo, hi);
    const float mi = fmaf(x, r, kMagic);
    const float e = fmaf(-(mi - kMagic), s, x);
    bad |= !(fabsf(e) < half);
    if (!IN_RANGE) bad |= v[i] != v[i];
    m[i] = __float_as_uint(mi);
  }
  if (bad) {
#pragma unroll
    for (int i = 0; i < N; ++i) m[i] = (uint32_t)(int)quant8_r(v[i], s, recip_or_zero(s));
  }
#pragma unroll
  for (int i = 0; i < N / 4; ++i) {
    // bytes [m0, m1, 0, 0] and [m2, m3, 0, 0], then the low halves side by side
    const uint32_t lo2 = __builtin_amdgcn_perm(m[4 * i + 1], m[4 * i], 0x0c0c0400u);
    const uint32_t hi2 = __builtin_amdgcn_perm(m[4 * i + 3], m[4 * i + 2], 0x0c0c0400u);
    w[i] = lo2 | (hi2 << 16);
  }
}

// x of the lane that differs in one bit of its number, for a reduction over 2, 4, 8 or 16 neighbouring
// lanes in that order (the mirrored rows hold equal values by then). STEP: that bit's value.
template <int STEP>
__device__ __forceinline__ float dpp_partner(float x) {
  constexpr int kCtrl = STEP == 1 ? 0xB1 : STEP == 2 ? 0x4E : STEP == 4 ? 0x141 : 0x140;
  return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, x), kCtrl, 0xF, 0xF, true));
}

// Wave-uniform value in an SGPR (so loads indexed by it can go through the scalar cache).
__device__ __forceinline__ int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }

}  // namespace qssm
