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
// as root mean squares over the output 1.4e-5 of it for normal data, 5e-5 for codes of every exponent, beside an fp16 y's
// own rounding of up to 2^-11 of each value. An fp32 y is worth more: there the codes are converted to fp16, exactly, for
// v_mfma_f32_32x32x16_f16, at half the rate, whose sums are off by 1e-8 to 6e-7.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <type_traits>

#include "common.hpp"
#include "gemm_f8_forms.hpp"
#include "sequences.hpp"

using namespace qssm;
using namespace qssm_f8;

namespace {

typedef int v4i __attribute__((ext_vector_type(4)));
typedef int v8i __attribute__((ext_vector_type(8)));
typedef _Float16 v2h __attribute__((ext_vector_type(2)));
typedef _Float16 v8h __attribute__((ext_vector_type(8)));
typedef float v4f __attribute__((ext_vector_type(4)));
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

// 16 codes of a row from k on, at any address (the hardware takes unaligned 16-byte loads); codes at or past K are 0 and
// not read. A chunk that reaches past K is the end of the row's last 16 codes, shifted into place without a
// branch, so that a thread's loads are in flight together; K >= 16 (load16_short: any K, byte by byte).
__device__ __forceinline__ uint4 load16(const uint8_t* row, int64_t k, int64_t K) {
  const int64_t at = min(k, K - 16);
  uint32_t w[4];
  __builtin_memcpy(w, row + at, 16);
  const int n = (int)min(k - at, (int64_t)16);
#pragma unroll
  for (int i = 0; i < 4; ++i) w[i] = (n & 16) ? 0u : w[i];
#pragma unroll
  for (int i = 0; i < 4; ++i) w[i] = (n & 8) ? (i < 2 ? w[(i + 2) & 3] : 0u) : w[i];
#pragma unroll
  for (int i = 0; i < 4; ++i) w[i] = (n & 4) ? (i < 3 ? w[(i + 1) & 3] : 0u) : w[i];
  const uint32_t b = n & 3;
  return make_uint4(__builtin_amdgcn_alignbyte(w[1], w[0], b), __builtin_amdgcn_alignbyte(w[2], w[1], b),
                    __builtin_amdgcn_alignbyte(w[3], w[2], b), __builtin_amdgcn_alignbyte(0u, w[3], b));
}

__device__ __forceinline__ uint4 load16_short(const uint8_t* row, int64_t k, int64_t K) {
  uint32_t w[4] = {0u, 0u, 0u, 0u};
#pragma unroll
  for (int i = 0; i < 16; ++i)
    if (k + i < K) w[i / 4] |= (uint32_t)row[k + i] << (8 * (i % 4));
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

typedef __attribute__((address_space(3))) void* lds_ptr;
constexpr int kBufferWord3 = 0x00020000;  // buffer resource word 3 for raw 32-bit access (gfx9)

// 16 (or 4) bytes per lane from byte voff + soff of the buffer straight to LDS, at dst (wave-uniform) + 16 (4) lane
__device__ __forceinline__ void load_lds(__amdgpu_buffer_rsrc_t r, uint8_t* dst, int voff, int soff) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_ptr)dst, 16, voff, soff, 0, 0);
}

__device__ __forceinline__ void load_lds_word(__amdgpu_buffer_rsrc_t r, uint8_t* dst, int voff, int soff) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_ptr)dst, 4, voff, soff, 0, 0);
}

__device__ __forceinline__ __amdgpu_buffer_rsrc_t rsrc_of(const void* p, int bytes = 0x7fffffff) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), (short)0, bytes, kBufferWord3);
}

// The activations' scales of block b from row m0 on (`rows` of them; behind those, zeros).
__device__ __forceinline__ __amdgpu_buffer_rsrc_t scales_of(const GemmParams& p, int b, int64_t m0, int rows) {
  return rsrc_of(p.sa + b * p.sas + m0, (int)min(p.M - m0, (int64_t)rows) * 4);
}

// Keeps the compiler's LDS accesses on their side (the direct loads are not its accesses).
__device__ __forceinline__ void fence() { asm volatile("" ::: "memory"); }

// Waits until at most N vector memory operations are outstanding, and for every LDS read.
// (vmcnt in bits 3:0 and 15:14, expcnt 6:4 not waited for, lgkmcnt 11:8)
template <int N>
__device__ __forceinline__ void wait_vm_lds() {
  static_assert(N <= 63, "vmcnt has 6 bits");
  fence();
  __builtin_amdgcn_s_waitcnt((N & 15) | ((N >> 4) << 14) | 0x70);
  fence();
}

__device__ __forceinline__ void to_type(float v, __half& o) { o = __float2half_rn(v); }
__device__ __forceinline__ void to_type(float v, float& o) { o = v; }

// The wave's 32 TM x 32 TN outputs from row mw, column nw: lane l holds row l % 32 and, in register 4 j + i, column
// 8 j + 4 (l / 32) + i. Each 32 rows are turned through the wave's part of LDS into whole-row stores. STREAM:
// stores that do not displace the operands from L2.
template <int TM, int TN, bool STREAM, typename T>
__device__ __forceinline__ void epilogue(const GemmParams& p, uint8_t* sm, const v16f (&acc)[TM][TN], int64_t mw, int64_t nw,
                                         int wave, int lane) {
  constexpr int kCols = TN * 32, kRowB = kCols * (int)sizeof(T) + 16, kPer = 16 / (int)sizeof(T);
  constexpr int kLanes = kCols / kPer;  // lanes per row of 16-byte stores
  uint8_t* buf = sm + wave * 32 * kRowB;
  const int kh = lane >> 5;
  T* y = reinterpret_cast<T*>(p.y);
  const bool vec = nw + kCols <= p.N && ((uintptr_t)p.y | (uintptr_t)(p.ys * (int64_t)sizeof(T))) % 16 == 0;
#pragma unroll
  for (int mt = 0; mt < TM; ++mt) {
#pragma unroll
    for (int nt = 0; nt < TN; ++nt)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int c = nt * 32 + 8 * j + 4 * kh;
        T o[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float b = p.bias ? p.bias[min(nw + c + i, p.N - 1)] : 0.0f;
          to_type(acc[mt][nt][4 * j + i] + b, o[i]);
        }
        __builtin_memcpy(__builtin_assume_aligned(buf + (lane & 31) * kRowB + c * sizeof(T), 8), o, 4 * sizeof(T));
      }
    wait_vm_lds<63>();  // the wave's own buffer: its LDS operations run in order
    const int64_t mb = mw + mt * 32;
    if (vec) {
#pragma unroll
      for (int r = 0; r < 32; r += 64 / kLanes) {
        const int row = r + lane / kLanes;
        const v4i v = *reinterpret_cast<const v4i*>(buf + row * kRowB + (lane % kLanes) * 16);
        v4i* dst = reinterpret_cast<v4i*>(y + (mb + row) * p.ys + nw + (lane % kLanes) * kPer);
        if (mb + row < p.M) {
          if (STREAM) __builtin_nontemporal_store(v, dst);
          else *dst = v;
        }
      }
    } else {
      constexpr int kStep = 64 / kCols > 0 ? 64 / kCols : 1, kLine = kCols < 64 ? kCols : 64;
#pragma unroll
      for (int c0 = 0; c0 < kCols; c0 += kLine) {
        const int c = c0 + lane % kLine;
        if (nw + c < p.N)
#pragma unroll 8
          for (int r = lane / kLine; r < 32; r += kStep)
            if (mb + r < p.M) y[(mb + r) * p.ys + nw + c] = reinterpret_cast<const T*>(buf + r * kRowB)[c];
      }
    }
    wait_vm_lds<63>();
  }
}

// ------------------------------------------------------------------------------------------------
// Tiles of (32 WM TM) x (32 WN TN) shared by WM x WN waves. K runs in steps of one scale block through NS LDS stages
// that direct loads fill NS steps ahead, with the rows' scales beside them; one barrier per step, placed where
// every wave has the step's last fragments in registers. A wave keeps the step's weight fragments and reads its
// activations' a row tile ahead, and the next step's under the last products. A tile's products of the block go
// to a sum of their own, which is scaled and added.
// The stages ahead are waited for earlier than the two stages need: the next step's weight scale is a vector load of every step,
// vector memory is waited for in order, and so with NS = 2 the wait before the barrier (all but (NS - 2) loads) holds for the
// load just issued, and the wait for the first scale, issued behind the first stages' loads, for nearly all of
// those, at the entry of the loop and so at its start in every turn. The costs in gemm_f8_forms.hpp hold with these waits.
// KG groups of waves take every KG-th step each, in stages of their own, and join their sums in LDS in the groups'
// order: where one workgroup has a CU, its step's latency bounds it (64x64 tiles, 256 x 4096 x 8192, fp16 y: 29
// us with one group, 23 with two, 22 with four).
// 16384 x 18560 x 4096 in 256x256 tiles: 1250 us (2.0 PFLOP/s). Without the scaled additions it takes 1063, without the
// reads of LDS 1085, without the direct loads 997 (at 1.6 GHz under its load): no single one bounds it, and
// holding a tile's sum back until the next one's products run, so that neither waits, gained nothing.
// The partial step of a K that is no multiple of 128 is the first and goes through registers, with zeros past K. Rows
// past M or N read the last row and are not stored.
// Tile order: 8 contiguous ranges, one per XCD, in groups of 4 row tiles, so that the workgroups that run together on an
// XCD share rows and columns in its L2.
template <int WM, int WN, int TM, int TN, int NS>
struct Tile {
  static constexpr int kWaves = WM * WN, kBM = WM * TM * 32, kBN = WN * TN * 32;
  static constexpr int kNA = kBM / 8 / kWaves, kNB = kBN / 8 / kWaves;  // loads of a wave, 8 rows each
  static constexpr int kPieces = (kBM + 63) / 64, kNX = (kPieces + kWaves - 1) / kWaves;  // loads of 64 rows' scales, some of them twice
  static constexpr int kCodes = (kBM + kBN) * 128, kStage = kCodes + kPieces * 256;
};

template <bool EXACT>
using Out = std::conditional_t<EXACT, float, __half>;

// First row and column of this workgroup's tile; false in the grid's padding (the whole workgroup).
__device__ __forceinline__ bool tile_of(const GemmParams& p, int bm, int bn, int64_t& m0, int64_t& n0) {
  const int64_t nm = (p.M + bm - 1) / bm, nn = (p.N + bn - 1) / bn;
  const int64_t id = (int64_t)(blockIdx.x % 8) * (gridDim.x / 8) + blockIdx.x / 8;
  if (id >= nm * nn) return false;
  constexpr int64_t kGM = 4;
  const int64_t grp = id / (kGM * nn), fm = grp * kGM;
  const int64_t gsz = min(nm - fm, kGM), within = id - grp * kGM * nn;
  m0 = (fm + within % gsz) * bm;
  n0 = (within / gsz) * bn;
  return true;
}

template <int WM, int WN, int TM, int TN, int NS, int KG, bool EXACT>
__global__ __launch_bounds__(WM * WN * KG * 64) void k_gemm_f8_tile(GemmParams p) {
  using G = Tile<WM, WN, TM, TN, NS>;
  constexpr int kLd = G::kNA + G::kNB + G::kNX;
  static_assert(TN * 32 <= 128, "a wave's columns lie in one block of the weights' scales");
  static_assert(TM % 2 == 0 || TM == 1, "the row tiles' fragments alternate between two sets");
  constexpr int kOutB = G::kWaves * 32 * (TN * 32 * (int)sizeof(Out<EXACT>) + 16);
  constexpr int kJoin = (KG - 1) * G::kWaves * TM * TN * 4096;
  __shared__ __align__(1024) uint8_t all[std::max({KG * NS * G::kStage, kOutB, kJoin})];
  const int tid = threadIdx.x, lane = tid & 63;
  const int group = uniform(tid >> 6) / G::kWaves, wave = uniform(tid >> 6) % G::kWaves;
  uint8_t* const sm = all + group * NS * G::kStage;
  const int wm = wave / WN, wn = wave % WN, kh = lane >> 5, l31 = lane & 31;
  int64_t m0, n0;
  if (!tile_of(p, G::kBM, G::kBN, m0, n0)) return;
  const uint8_t* abase = p.a + m0 * p.as;
  const uint8_t* wbase = p.w + n0 * p.ws;
  const int alast = (int)min(p.M - 1 - m0, (int64_t)G::kBM), wlast = (int)min(p.N - 1 - n0, (int64_t)G::kBN);
  // load i of this wave: 8 rows, lane l at row l / 8, slot l % 8 (32-bit offsets: host)
  int aoff[G::kNA], woff[G::kNB];
#pragma unroll
  for (int i = 0; i < G::kNA; ++i) {
    const int row = (wave * G::kNA + i) * 8 + lane / 8;
    aoff[i] = min(row, alast) * (int)p.as + (lane % 8 ^ swizzle(row)) * 16;
  }
#pragma unroll
  for (int i = 0; i < G::kNB; ++i) {
    const int row = (wave * G::kNB + i) * 8 + lane / 8;
    woff[i] = min(row, wlast) * (int)p.ws + (lane % 8 ^ swizzle(row)) * 16;
  }
  const int full = (int)(p.K / 128), tail = (int)(p.K % 128) != 0, nsteps = full + tail;  // host: full >= 1
  const int count = (nsteps + KG - 1) / KG;  // steps of a group: group, group + KG, ...
  const __amdgpu_buffer_rsrc_t ra = rsrc_of(abase), rw = rsrc_of(wbase);
  uint8_t* dst_a = sm + wave * G::kNA * 1024;
  uint8_t* dst_w = sm + G::kBM * 128 + wave * G::kNB * 1024;
  const auto step_of = [&](int s) { return min(s * KG + group, nsteps - 1); };
  const auto block_of = [&](int s) { return step_of(s) < tail ? full : step_of(s) - tail; };

  // the group's step s into stage st; past the last step the last one again, so that the waits stay exact
  const auto issue_scales = [&](int s, int st) {
    const __amdgpu_buffer_rsrc_t rs = scales_of(p, block_of(s), m0, G::kBM);
#pragma unroll
    for (int i = 0; i < G::kNX; ++i) {
      const int row = (wave * G::kNX + i) % G::kPieces * 64;
      load_lds_word(rs, sm + st * G::kStage + G::kCodes + row * 4, lane * 4, row * 4);
    }
  };
  const auto issue = [&](int s, int st) {
    const int koff = (step_of(s) - tail) * 128;
#pragma unroll
    for (int i = 0; i < G::kNA; ++i) load_lds(ra, dst_a + st * G::kStage + i * 1024, aoff[i], koff);
#pragma unroll
    for (int i = 0; i < G::kNB; ++i) load_lds(rw, dst_w + st * G::kStage + i * 1024, woff[i], koff);
    issue_scales(s, st);
  };

  v16f acc[TM][TN];
#pragma unroll
  for (int mt = 0; mt < TM; ++mt)
#pragma unroll
    for (int nt = 0; nt < TN; ++nt) acc[mt][nt] = v16f{};
  v8i fa[2][2], fb[TN][2];  // [set][slice], [column tile][slice]
  const auto read_a = [&](int st, int mt, int set) {
#pragma unroll
    for (int ks = 0; ks < 2; ++ks) fa[set][ks] = fragment(sm + st * G::kStage, (wm * TM + mt) * 32 + l31, ks, kh);
  };
  const auto read_b = [&](int st, int nt) {
#pragma unroll
    for (int ks = 0; ks < 2; ++ks) fb[nt][ks] = fragment(sm + st * G::kStage, G::kBM + (wn * TN + nt) * 32 + l31, ks, kh);
  };
  float sa[TM];
  const auto read_scales = [&](int st) {
    const float* at = reinterpret_cast<const float*>(sm + st * G::kStage + G::kCodes) + wm * TM * 32 + l31;
#pragma unroll
    for (int mt = 0; mt < TM; ++mt) sa[mt] = at[mt * 32];
  };
  const float* swrow = p.sw + min(n0 + wn * TN * 32, p.N - 1) / 128 * p.kb;

  const bool part_first = tail && group == 0;
  if (!part_first) issue(0, 0);
#pragma unroll
  for (int d = 1; d < NS; ++d) issue(d, d);
  if (part_first) {
    issue_scales(0, 0);
    uint4 va[G::kNA], vw[G::kNB];
#pragma unroll
    for (int i = 0; i < G::kNA; ++i) {
      const int row = (wave * G::kNA + i) * 8 + lane / 8;
      va[i] = load16(abase + (int64_t)min(row, alast) * p.as, (int64_t)full * 128 + (lane % 8 ^ swizzle(row)) * 16, p.K);
    }
#pragma unroll
    for (int i = 0; i < G::kNB; ++i) {
      const int row = (wave * G::kNB + i) * 8 + lane / 8;
      vw[i] = load16(wbase + (int64_t)min(row, wlast) * p.ws, (int64_t)full * 128 + (lane % 8 ^ swizzle(row)) * 16, p.K);
    }
#pragma unroll
    for (int i = 0; i < G::kNA; ++i) *reinterpret_cast<uint4*>(dst_a + i * 1024 + lane * 16) = va[i];
#pragma unroll
    for (int i = 0; i < G::kNB; ++i) *reinterpret_cast<uint4*>(dst_w + i * 1024 + lane * 16) = vw[i];
    wait_vm_lds<0>();
  }
  wait_vm_lds<(NS - 1) * kLd>();
  __builtin_amdgcn_s_barrier();
  fence();
#pragma unroll
  for (int nt = 0; nt < TN; ++nt) read_b(0, nt);
  read_a(0, 0, 0);
  read_scales(0);
  float sw = swrow[block_of(0)];
  int st = 0, s = 0;
  // a step; ODD: its first row tile's fragments are in set TM % 2
  const auto step = [&](auto odd) {
    constexpr int kFirst = decltype(odd)::value ? TM % 2 : 0;
    const int nx = st + 1 == NS ? 0 : st + 1;
    const float sw_next = swrow[block_of(s + 1)];
    const float w = s * KG + group < nsteps ? valid_or_zero(sw) : 0.0f;
    float sc[TM];
#pragma unroll
    for (int mt = 0; mt < TM; ++mt) sc[mt] = valid_or_zero(sa[mt]) * w;
#pragma unroll
    for (int mt = 0; mt < TM; ++mt) {
      const bool last = mt + 1 == TM;
      const int set = (kFirst + mt) & 1;
      if (last) {
        // every wave has the last fragments of stage st in registers, and step s + 1 has landed
        wait_vm_lds<(NS - 2) * kLd>();
        __builtin_amdgcn_s_barrier();
        fence();
        issue(s + NS, st);
      }
      read_a(last ? nx : st, last ? 0 : mt + 1, set ^ 1);
      v16f part[TN];
#pragma unroll
      for (int nt = 0; nt < TN; ++nt) {
        part[nt] = product<EXACT>(fb[nt][0], fa[set][0], v16f{});
        part[nt] = product<EXACT>(fb[nt][1], fa[set][1], part[nt]);
        if (last) read_b(nx, nt);  // the next step's, while the sums below are added
      }
      if (last) read_scales(nx);
#pragma unroll
      for (int nt = 0; nt < TN; ++nt)
#pragma unroll
        for (int i = 0; i < 16; ++i) acc[mt][nt][i] = fmaf(part[nt][i], sc[mt], acc[mt][nt][i]);
    }
    sw = sw_next;
    st = nx;
    ++s;
  };
  // (twice: one row tile's fragments alternate between the sets; for two row tiles it saves 4 %, for four it costs registers)
  if constexpr (TM > 2) {
    while (s < count) step(std::false_type());
  } else {
    while (s + 1 < count) {
      step(std::false_type());
      step(std::true_type());
    }
    if (s < count) step(std::false_type());
  }
  wait_vm_lds<0>();  // no direct load outlives the stages it writes
  __syncthreads();   // every wave is done with them: they become the buffers of what follows
  if constexpr (KG > 1) {
    float* join = reinterpret_cast<float*>(all) + wave * TM * TN * 1024 + lane;
    if (group > 0) {
#pragma unroll
      for (int t = 0; t < TM * TN; ++t)
#pragma unroll
        for (int i = 0; i < 16; ++i) join[(group - 1) * G::kWaves * TM * TN * 1024 + t * 1024 + i * 64] = acc[t / TN][t % TN][i];
    }
    __syncthreads();
    if (group == 0) {
#pragma unroll
      for (int g = 1; g < KG; ++g)
#pragma unroll
        for (int t = 0; t < TM * TN; ++t)
#pragma unroll
          for (int i = 0; i < 16; ++i) acc[t / TN][t % TN][i] += join[(g - 1) * G::kWaves * TM * TN * 1024 + t * 1024 + i * 64];
    }
    __syncthreads();
    if (group > 0) return;
  }
  epilogue<TM, TN, G::kBM == 256, Out<EXACT>>(p, all, acc, m0 + wm * TM * 32, n0 + wn * TN * 32, wave, lane);
}

// Tiles of 64 x 64, a quarter a wave, with the operands through registers: rows at any address, any K.
template <bool EXACT, bool SHORT>
__global__ __launch_bounds__(256) void k_gemm_f8_any(GemmParams p) {
  constexpr auto load_chunk = SHORT ? load16_short : load16;
  __shared__ __align__(16) uint8_t sm[2][2][64 * 128];
  const int tid = threadIdx.x, lane = tid & 63, wave = uniform(tid >> 6), kh = lane >> 5;
  int64_t m0, n0;
  if (!tile_of(p, 64, 64, m0, n0)) return;
  const int wm = wave & 1, wn = wave >> 1;
  const int64_t m = m0 + wm * 32 + (lane & 31), mc = min(m, p.M - 1);
  const float* sw = p.sw + n0 / 128 * p.kb;
  uint4 va[2], vw[2];
  const auto load = [&](int b) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int row = (tid + 256 * i) / 8, c = tid % 8;
      va[i] = load_chunk(p.a + min(m0 + row, p.M - 1) * p.as, (int64_t)b * 128 + c * 16, p.K);
      vw[i] = load_chunk(p.w + min(n0 + row, p.N - 1) * p.ws, (int64_t)b * 128 + c * 16, p.K);
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
  v16f acc[1][1] = {{v16f{}}};
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
    for (int i = 0; i < 16; ++i) acc[0][0][i] = fmaf(part[i], s, acc[0][0][i]);
    if (b + 1 < p.kb) store((b + 1) & 1);
  }
  __syncthreads();  // the stages become the waves' output buffers
  epilogue<1, 1, false, Out<EXACT>>(p, &sm[0][0][0], acc, m0 + wm * 32, n0 + wn * 32, wave, lane);
}

// ------------------------------------------------------------------------------------------------
// Up to 16 tokens: bound by the bytes of the weights, which go straight to registers, kDeep blocks ahead. A workgroup owns 16
// output channels, its W waves each W-th block of K; their sums are joined in LDS in the waves' order. Lane l
// holds row l % 16 and the 16 codes at 16 (l / 16) and at 64 + 16 (l / 16) of a block, so that a load's lanes cover whole
// 64-byte pieces; any address and any K.
template <bool EXACT, int W, int kDeep>
__global__ __launch_bounds__(W * 64) void k_gemm_f8_few(GemmParams p) {
  __shared__ v4f sums[W][64];
  const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6), q = lane >> 4;
  const int64_t n0 = (int64_t)blockIdx.x * 16;
  const int m = lane & 15;
  const uint8_t* a = p.a + (int64_t)min((int64_t)m, p.M - 1) * p.as + q * 16;
  const uint8_t* w = p.w + min(n0 + m, p.N - 1) * p.ws + q * 16;
  const float* sa = p.sa + min((int64_t)m, p.M - 1);
  const float* sw = p.sw + n0 / 128 * p.kb;
  const int full = (int)(p.K / 128);
  v4i va[kDeep][2], vw[kDeep][2];
  float s[kDeep];
  const auto load = [&](int b, int at) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      __builtin_memcpy(&vw[at][h], w + (int64_t)b * 128 + h * 64, 16);
      __builtin_memcpy(&va[at][h], a + (int64_t)b * 128 + h * 64, 16);
    }
    s[at] = sa[b * p.sas];
  };
  v4f acc = v4f{};
  const auto add = [&](int b, const v4i (&fw)[2], const v4i (&fa)[2], float scale) {
    const float by = valid_or_zero(scale) * valid_or_zero(sw[b]);
    v4f d = v4f{};
    if constexpr (EXACT) {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        d = __builtin_amdgcn_mfma_f32_16x16x32_f16(to_half(fw[i / 2][2 * (i % 2)], fw[i / 2][2 * (i % 2) + 1]),
                                                   to_half(fa[i / 2][2 * (i % 2)], fa[i / 2][2 * (i % 2) + 1]), d, 0, 0, 0);
    } else {
      d = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(__builtin_shufflevector(fw[0], fw[1], 0, 1, 2, 3, 4, 5, 6, 7),
                                                           __builtin_shufflevector(fa[0], fa[1], 0, 1, 2, 3, 4, 5, 6, 7), d, 0, 0, 0, 0, 0, 0);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[i] = fmaf(d[i], by, acc[i]);
  };
#pragma unroll
  for (int d = 0; d < kDeep; ++d)
    if (wave + d * W < full) load(wave + d * W, d);
  for (int b = wave; b < full; b += kDeep * W) {
#pragma unroll
    for (int d = 0; d < kDeep; ++d)
      if (b + d * W < full) {
        add(b + d * W, vw[d], va[d], s[d]);
        if (b + (d + kDeep) * W < full) load(b + (d + kDeep) * W, d);
      }
  }
  if (full < p.kb && wave == full % W) {
    v4i fw[2], fa[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const auto chunk = [&](const uint8_t* row) {
        const int64_t k = (int64_t)full * 128 + h * 64 + q * 16;
        return __builtin_bit_cast(v4i, p.K < 16 ? load16_short(row - q * 16, k, p.K) : load16(row - q * 16, k, p.K));
      };
      fw[h] = chunk(w);
      fa[h] = chunk(a);
    }
    add(full, fw, fa, sa[full * p.sas]);
  }
  sums[wave][lane] = acc;
  __syncthreads();
  if (wave != 0) return;
#pragma unroll
  for (int k = 1; k < W; ++k) acc += sums[k][lane];
  if (m >= p.M) return;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int64_t n = n0 + 4 * q + i;
    if (n < p.N) put(p, m, n, acc[i] + (p.bias ? p.bias[n] : 0.0f));
  }
}

unsigned grid_of(const GemmParams& p, int bm, int bn) { return (unsigned)(cdiv(cdiv(p.M, bm) * cdiv(p.N, bn), 8) * 8); }

template <bool EXACT>
void launch(const GemmParams& p, hipStream_t stream) {
  // up to 16 tokens: 1 x 18560 x 4096 fp16 16 us (19 in 64x64 tiles), 16 x 18560 x 4096 21 (19), 16 x 4096 x 8192 10 (12 in 32x32)
  if (p.M <= 16 && cdiv(p.N, 16) < kMaxTiles) {
    k_gemm_f8_few<EXACT, 8, 4><<<(unsigned)cdiv(p.N, 16), 512, 0, stream>>>(p);
    return;
  }
  // direct loads to LDS take multiples of 4 bytes, and whole blocks
  if (((uintptr_t)p.a | (uintptr_t)p.w | (uintptr_t)p.as | (uintptr_t)p.ws) % 4 != 0 || p.K < 128) {
    // (128x128 tiles that load alike leave one wave to a SIMD: 4096 x 4095 x 4097 349 us, 265 in these)
    const unsigned grid = grid_of(p, 64, 64);
    if (p.K < 16) k_gemm_f8_any<EXACT, true><<<grid, 256, 0, stream>>>(p);
    else k_gemm_f8_any<EXACT, false><<<grid, 256, 0, stream>>>(p);
    return;
  }
  switch (choose_form(p.M, p.N, p.K, !EXACT)) {
    case TILE256:
      if constexpr (!EXACT) k_gemm_f8_tile<2, 4, 4, 2, 2, 1, EXACT><<<grid_of(p, 256, 256), 512, 0, stream>>>(p);
      break;
    case TILE128: k_gemm_f8_tile<2, 2, 2, 2, 2, 1, EXACT><<<grid_of(p, 128, 128), 256, 0, stream>>>(p); break;
    case TILE64: k_gemm_f8_tile<2, 2, 1, 1, 3, 1, EXACT><<<grid_of(p, 64, 64), 256, 0, stream>>>(p); break;
    case TILE64K2: k_gemm_f8_tile<2, 2, 1, 1, 3, 2, EXACT><<<grid_of(p, 64, 64), 512, 0, stream>>>(p); break;
    case TILE64K4: k_gemm_f8_tile<2, 2, 1, 1, 2, 4, EXACT><<<grid_of(p, 64, 64), 1024, 0, stream>>>(p); break;
    case TILE32K4: k_gemm_f8_tile<1, 1, 1, 1, 2, 4, EXACT><<<grid_of(p, 32, 32), 256, 0, stream>>>(p); break;
    case TILE32K4DEEP: k_gemm_f8_tile<1, 1, 1, 1, 4, 4, EXACT><<<grid_of(p, 32, 32), 256, 0, stream>>>(p); break;
    default: k_gemm_f8_tile<4, 2, 2, 2, 2, 1, EXACT><<<grid_of(p, 256, 128), 512, 0, stream>>>(p);
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
  if (cdiv(M, 64) * cdiv(N, 64) >= (1 << 24) - 8) return fail(QSSM_ERR_UNSUPPORTED, "M * N too large");
  const Span y{a->y, M, a->y_stride * sy, N * sy};
  if (overlap(y, Span{a->a, M, a->a_stride, K}) || overlap(y, Span{a->w, N, a->w_stride, K}) || overlap(y, flat(a->bias, N * 4)) ||
      overlap(y, Span{a->a_scales, kb, a->a_scales_stride * 4, M * 4}) || overlap(y, flat(a->w_scales, cdiv(N, 128) * kb * 4)))
    return fail(QSSM_ERR_INVALID_ARG, "y overlaps an input");
  const GemmParams p{M, N, K, a->a, a->a_stride, a->a_scales, a->a_scales_stride, a->w, a->w_stride, a->w_scales, a->bias, a->y,
                     a->y_stride, a->y_dtype == QSSM_F16, (int32_t)kb};
  p.yf16 ? launch<false>(p, stream) : launch<true>(p, stream);
  return launch_status("gemm_f8");
}
