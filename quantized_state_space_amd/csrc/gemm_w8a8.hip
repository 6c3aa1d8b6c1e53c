// W8A8 linear layer: int8 weights x int8 activations on int8 MFMA with int32 accumulation.
//
// Quamba2, abstract: W8A8 blocks, prefill and generation (the in and out projections around the
// recurrence).
//     y[m, n] = bias[n] + sa[m] sw[n] * sum_k a[m, k] w[n, k]      (roundings: scaled())
// Both operands have k contiguous, which is the operand order of v_mfma_i32_32x32x32_i8: lane l of a
// wave holds row (or column) l % 32 and the 16 consecutive k at 16 (l / 32). The weights go in as the
// first operand, so a lane ends with one token and groups of 4 consecutive output channels.
//
// Tiles shared by a workgroup's waves with K in common steps (k_gemm_w8a8_tile, with a variant for rows
// at any address), and the smallest tiles with K split over the waves (k_gemm_w8a8_split: few tokens,
// bound by the bytes of the weights and by latency). choose_form() picks by estimated time.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <type_traits>

#include "common.hpp"
#include "gemm_w8a8_forms.hpp"

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
// of the scales, one of the fused multiply-add (and one more to an fp16 y).
__device__ __forceinline__ float scaled(float sa, float sw, int acc, float bias) {
  return fmaf(sa * sw, (float)acc, bias);
}

// s in [2^-63, 2^63], by its bits: the product of two such scales is a normal fp32 number.
__device__ __forceinline__ bool tame(float s) { return __float_as_uint(s) - 0x20000000u <= 0x3f000000u; }

// The same for any valid scales (2^-100 to 2^100) and the 0 of one that is not: a product that may be an
// infinity, a 0 or a few bits in fp32 is taken in fp64, where it is exact, and the result rounds once.
__device__ __forceinline__ float scaled_wide(float sa, float sw, int acc, float bias) {
  if (tame(sa) && tame(sw)) return scaled(sa, sw, acc, bias);
  return (float)fma((double)sa * (double)sw, (double)acc, (double)bias);
}

__device__ __forceinline__ void put(const GemmParams& p, int64_t m, int64_t n, float v) {
  if (p.yf16) reinterpret_cast<__half*>(p.y)[m * p.ys + n] = __float2half_rn(v);
  else reinterpret_cast<float*>(p.y)[m * p.ys + n] = v;
}

// 16 consecutive codes of a row of K from k on, at any alignment (the hardware takes unaligned 16-byte
// loads); codes at or past K are 0 and not read. A chunk that reaches past K is the end of the row's last
// 16 codes, shifted into place without a branch, so that a thread's loads are in flight together; K >= 16
// (load16_short: any K, byte by byte, a load and a wait each).
__device__ __forceinline__ uint4 load16(const int8_t* row, int64_t k, int64_t K) {
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

__device__ __forceinline__ uint4 load16_short(const int8_t* row, int64_t k, int64_t K) {
  uint32_t w[4] = {0u, 0u, 0u, 0u};
#pragma unroll
  for (int i = 0; i < 16; ++i)
    if (k + i < K) w[i / 4] |= (uint32_t)(uint8_t)row[k + i] << (8 * (i % 4));
  return make_uint4(w[0], w[1], w[2], w[3]);
}

typedef __attribute__((address_space(3))) void* lds_ptr;
constexpr int kBufferWord3 = 0x00020000;  // buffer resource word 3 for raw 32-bit access (gfx9)

// 16 bytes per lane from byte voff + soff of the buffer straight to LDS, at dst (wave-uniform) + 16 lane
__device__ __forceinline__ void load_lds(__amdgpu_buffer_rsrc_t r, int8_t* dst, int voff, int soff) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_ptr)dst, 16, voff, soff, 0, 0);
}

// 4 bytes per lane, at dst + 4 lane
__device__ __forceinline__ void load_lds_word(__amdgpu_buffer_rsrc_t r, int8_t* dst, int voff, int soff) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_ptr)dst, 4, voff, soff, 0, 0);
}

// The 16 codes from byte sh on of v and the word behind it.
__device__ __forceinline__ v4i shifted(const v4i& v, uint32_t next, uint32_t sh) {
  return v4i{(int)__builtin_amdgcn_alignbyte(v[1], v[0], sh), (int)__builtin_amdgcn_alignbyte(v[2], v[1], sh),
             (int)__builtin_amdgcn_alignbyte(v[3], v[2], sh), (int)__builtin_amdgcn_alignbyte(next, v[3], sh)};
}

// The word behind the partial step that follows `full` steps of BK bytes, of K bytes from `row` (a
// multiple of 4) on: it holds at most three codes, and is read where it holds any (else the row's first).
template <int BK>
__device__ __forceinline__ uint32_t word_behind(const int8_t* row, int full, int64_t K) {
  const int left = (int)K - (full + 1) * BK;
  const uint32_t w = *reinterpret_cast<const uint32_t*>(row + (left > 0 ? (full + 1) * BK : 0));
  return left > 0 ? w & ((1u << (8 * left)) - 1u) : 0u;
}

__device__ __forceinline__ __amdgpu_buffer_rsrc_t rsrc_of(const int8_t* p, int bytes = 0x7fffffff) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<int8_t*>(p), (short)0, bytes, kBufferWord3);
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

template <int N>
__device__ __forceinline__ void wait_vm() {
  static_assert(N <= 63, "vmcnt has 6 bits");
  fence();
  __builtin_amdgcn_s_waitcnt((N & 15) | ((N >> 4) << 14) | 0xF70);
  fence();
}

// LDS rows of 128 bytes; the 16-byte chunk c of row r is in slot c ^ swizzle(r), which spreads the rows
// that a 16-byte read serves together over all 64 banks (measured: no conflicts; 4 of 8 cycles of
// every read without it).
__device__ __forceinline__ int swizzle(int row) { return (row >> 1) & 7; }

// ------------------------------------------------------------------------------------------------
// Tiles of (32 WM TM) x (32 WN TN) shared by WM x WN waves. K runs in steps of BK bytes through NS LDS
// stages that direct loads fill NS - 1 steps ahead; one barrier per step, placed where every wave has
// the step's last fragments in registers, so that the last slice's products hide it. Fragments are
// read AHEAD slices of 32 codes ahead, and reads and loads are issued between the products.
// AHEAD > 1 (small tiles, whose products are too few to cover an LDS read): the barrier then stands
// where the fragments pass to the next step, and its step refills the stage before last; it pays with
// many stages, which leave room for one tile per CU (256 x 4096 x 8192 in 64x64 tiles: 18.1 us with 3
// stages, 18.1 with 6, 16.0 with 6 and AHEAD 3).
// Steps of 128 and few stages beat steps of 64 and twice the stages (half the barriers): 256x256 tiles,
// 16384 x 18560 x 4096: 1069 us (2.33 POPS) and 1128; 128x64 tiles, 256 x 4096 x 8192: 22 and 27.
// The many-token forms are bound by the power the matrix cores draw: with all operands 0 the same
// kernel takes 0.71 of the time (4096 x 4096 x 16384), and its clock under load is 1.4 GHz.
// The partial step of a K that is no multiple of BK is the first and goes through registers, with
// zeros past K. Rows past M or N read the last row and are not stored.
// Tile order: the tiles are cut into 8 contiguous ranges, one per XCD (workgroups are dealt to the
// XCDs in turn), in groups of 4 row tiles, so the workgroups that run together on an XCD share rows
// and columns in its L2 (16384 x 18560 x 4096: groups of 4 / 8 / 16 take 1029 / 1033 / 1049 us).
// SHIFT: rows at any address, K of any length. Direct loads take multiples of 4 bytes, so a row lies in
// LDS from the word on that holds its first code, 0 to 3 codes late, with the word behind each step's
// BK bytes beside the stage; a fragment is its 16 bytes and the next word shifted into place (the sums
// pair codes of the same k). 4096 x 4095 x 4097, fp32 y: 93 us, 77 with K = 4100 and no shift; fp16 y: 88, and 123
// with the operands through registers in place of direct loads (16384 x 9001 x 4001: 762 and 1048).
// Output: each wave scales its sums and turns 32 rows at a time through LDS into whole-row stores
// (stores straight from the registers took 23 us a tile, a third of the whole at K = 4096).
template <int WM, int WN, int TM, int TN, int NS, int BK, bool SHIFT = false>
struct Tile {
  static constexpr int kWaves = WM * WN, kBM = WM * TM * 32, kBN = WN * TN * 32, kRpl = 1024 / BK;
  static constexpr int kNA = kBM / kRpl / kWaves, kNB = kBN / kRpl / kWaves;  // loads of a wave, kRpl rows each
  static constexpr int kRows = kBM + kBN, kStage = kRows * (BK + (SHIFT ? 4 : 0));
  static constexpr int kNX = SHIFT ? (kRows / 64 + kWaves - 1) / kWaves : 0;  // loads of next words, 64 rows each
};

__device__ __forceinline__ void to_type(float v, __half& o) { o = __float2half_rn(v); }
__device__ __forceinline__ void to_type(float v, float& o) { o = v; }

// The wave's TM x TN tiles: lane l holds row l % 32 and, in register 4 j + i, column
// 8 j + 4 (l / 32) + i. STREAM (the forms for large y): stores that do not displace the operands from
// L2 (16384 x 18560 x 4096: 1029 us, 1096 without). WIDE: some of the wave's scales are not tame(); a form of its
// own, so that the usual one carries none of its code.
template <bool WIDE, int TM, int TN, bool STREAM, typename T>
__device__ __forceinline__ void epilogue(const GemmParams& p, int8_t* sm, const float* s_sw, const float* s_bias,
                                         const v16i (&acc)[TM][TN], const float (&sa)[TM], int64_t mw, int64_t nw,
                                         int wave, int lane) {
  constexpr int kCols = TN * 32, kRowB = kCols * (int)sizeof(T) + 16, kPer = 16 / (int)sizeof(T);
  constexpr int kLanes = kCols / kPer;  // lanes per row of 16-byte stores
  int8_t* buf = sm + wave * 32 * kRowB;
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
        const float4 sw = *reinterpret_cast<const float4*>(s_sw + c), bn = *reinterpret_cast<const float4*>(s_bias + c);
        const v16i& d = acc[mt][nt];
        T o[4];
        constexpr auto f = WIDE ? scaled_wide : scaled;
        to_type(f(sa[mt], sw.x, d[4 * j], bn.x), o[0]);
        to_type(f(sa[mt], sw.y, d[4 * j + 1], bn.y), o[1]);
        to_type(f(sa[mt], sw.z, d[4 * j + 2], bn.z), o[2]);
        to_type(f(sa[mt], sw.w, d[4 * j + 3], bn.w), o[3]);
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
      // 64 / kCols rows at a time, one element per lane
      constexpr int kStep = 64 / kCols;
      const int c = lane % kCols;
      T* dst = y + (mb + lane / kCols) * p.ys + nw + c;
      const T* src = reinterpret_cast<const T*>(buf + (lane / kCols) * kRowB) + c;
      if (nw + c < p.N) {
        if (mb + 32 <= p.M) {
#pragma unroll 8
          for (int r = 0; r < 32; r += kStep) dst[r * p.ys] = src[r * (kRowB / (int)sizeof(T))];
        } else {
          for (int r = 0; r < 32; r += kStep)
            if (mb + r + lane / kCols < p.M) dst[r * p.ys] = src[r * (kRowB / (int)sizeof(T))];
        }
      }
    }
    wait_vm_lds<63>();
  }
}

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

// The tile's column scales and biases to LDS, and the scales of the wave's rows (from row mw).
template <int TM>
__device__ __forceinline__ void load_scales(const GemmParams& p, int bn, int64_t mw, int64_t n0, int lane, int tid,
                                            int threads, float* s_sw, float* s_bias, float (&sa)[TM]) {
  for (int i = tid; i < bn; i += threads) {
    const int64_t n = min(n0 + i, p.N - 1);
    s_sw[i] = valid_or_zero(p.w_scales[n]);
    s_bias[i] = p.bias ? p.bias[n] : 0.0f;
  }
#pragma unroll
  for (int mt = 0; mt < TM; ++mt) {
    const int64_t m = min(mw + mt * 32 + (lane & 31), p.M - 1);
    sa[mt] = valid_or_zero(p.a_scales[p.per_row ? m : 0]);
  }
}

template <int WM, int WN, int TM, int TN, int NS, int BK, int AHEAD, bool SHIFT>
__global__ __launch_bounds__(WM * WN * 64) void k_gemm_w8a8_tile(GemmParams p) {
  using G = Tile<WM, WN, TM, TN, NS, BK, SHIFT>;
  constexpr int kLd = G::kNA + G::kNB + G::kNX, kSlots = BK / 16, kSlices = BK / 32;
  static_assert(WM * WN * 32 * (TN * 32 * 4 + 16) <= NS * G::kStage, "the output buffers fit the stages");
  // one array: with several the compiler waits for all direct loads before every LDS read
  __shared__ __align__(1024) int8_t sm[NS * G::kStage + 8 * G::kBN];
  float* s_sw = reinterpret_cast<float*>(sm + NS * G::kStage);
  float* s_bias = s_sw + G::kBN;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = uniform(tid >> 6);
  const int wm = wave / WN, wn = wave % WN, kh = lane >> 5;
  int64_t m0, n0;
  if (!tile_of(p, G::kBM, G::kBN, m0, n0)) return;
  float sa[TM];
  load_scales<TM>(p, G::kBN, m0 + wm * TM * 32, n0, lane, tid, G::kWaves * 64, s_sw, s_bias, sa);
  // load i of this wave: kRpl rows, lane l at row l / kSlots, slot l % kSlots (32-bit offsets: host)
  // (SHIFT: from the word that holds the row's first code on)
  const int8_t* abase = p.a + m0 * p.as;
  const int8_t* wbase = p.w + n0 * p.ws;
  const int apre = SHIFT ? (int)((uintptr_t)abase & 3) : 0, wpre = SHIFT ? (int)((uintptr_t)wbase & 3) : 0;
  abase -= apre;
  wbase -= wpre;
  constexpr int kWord = SHIFT ? ~3 : ~0;
  const int alast = (int)min(p.M - 1 - m0, (int64_t)G::kBM), wlast = (int)min(p.N - 1 - n0, (int64_t)G::kBN);
  const int as = (int)p.as, ws = (int)p.ws;
  const auto a_at = [&](int row) { return min(row, alast) * as + apre; };
  const auto w_at = [&](int row) { return min(row, wlast) * ws + wpre; };
  const int lrow = lane / kSlots;
  int aoff[G::kNA], woff[G::kNB], achk[G::kNA], wchk[G::kNB];
  uint32_t atail[G::kNA], wtail[G::kNB];  // codes before the row's first
#pragma unroll
  for (int i = 0; i < G::kNA; ++i) {
    const int row = (wave * G::kNA + i) * G::kRpl + lrow;
    achk[i] = ((lane % kSlots) ^ swizzle(row)) * 16;
    aoff[i] = a_at(row) & kWord;
    atail[i] = a_at(row) & ~kWord;
  }
#pragma unroll
  for (int i = 0; i < G::kNB; ++i) {
    const int row = (wave * G::kNB + i) * G::kRpl + lrow;
    wchk[i] = ((lane % kSlots) ^ swizzle(row)) * 16;
    woff[i] = w_at(row) & kWord;
    wtail[i] = w_at(row) & ~kWord;
  }
  // SHIFT: the word behind each row's BK bytes of a step; of rows that need none, the last one before
  int xoff[G::kNX + 1], xrow[G::kNX + 1];
  uint32_t xsh[G::kNX + 1];
#pragma unroll
  for (int i = 0; i < G::kNX; ++i) {
    xrow[i] = (wave * G::kNX + i) % (G::kRows / 64) * 64;
    const int row = xrow[i] + lane, at = xrow[i] < G::kBM ? a_at(row) : w_at(row - G::kBM);
    xsh[i] = at & 3;
    xoff[i] = (at & ~3) + BK - (xsh[i] ? 0 : 4);
  }
  const int full = (int)(p.K / BK), tail = (int)(p.K % BK) != 0;  // host: full >= 1 without SHIFT
  // without a full step every direct load is out of range: it reads nothing
  const int bytes = SHIFT && full == 0 ? 0 : 0x7fffffff;
  const __amdgpu_buffer_rsrc_t ra = rsrc_of(abase, bytes), rw = rsrc_of(wbase, bytes);
  const int nsteps = full + tail;
  int8_t* dst_a = sm + wave * G::kNA * 1024;
  int8_t* dst_w = sm + G::kBM * BK + wave * G::kNB * 1024;

  // step s into stage st; past the last step the last one again, so that the waits stay exact
  auto issue = [&](int s, int st) {
    const int koff = (SHIFT ? max(min(s, nsteps - 1) - tail, 0) : min(s, nsteps - 1) - tail) * BK;
#pragma unroll
    for (int i = 0; i < G::kNA; ++i) load_lds(ra, dst_a + st * G::kStage + i * 1024, aoff[i] + achk[i], koff);
#pragma unroll
    for (int i = 0; i < G::kNB; ++i) load_lds(rw, dst_w + st * G::kStage + i * 1024, woff[i] + wchk[i], koff);
#pragma unroll
    for (int i = 0; i < G::kNX; ++i)
      load_lds_word(xrow[i] < G::kBM ? ra : rw, sm + st * G::kStage + G::kRows * BK + xrow[i] * 4, xoff[i], koff);
  };

  v16i acc[TM][TN];
#pragma unroll
  for (int mt = 0; mt < TM; ++mt)
#pragma unroll
    for (int nt = 0; nt < TN; ++nt) acc[mt][nt] = v16i{};
  constexpr int kSets = AHEAD == 1 ? 2 : kSlices;
  v4i fa[kSets][TM], fb[kSets][TN];
  const int slot0 = (kh ^ swizzle(lane & 31)) * 16;
  const int arow = (wm * TM * 32 + (lane & 31)) * BK, brow = (G::kBM + wn * TN * 32 + (lane & 31)) * BK;
  [[maybe_unused]] uint32_t na[kSets][TM], nb[kSets][TN], sha[TM], shb[TN];
  if constexpr (SHIFT) {
#pragma unroll
    for (int mt = 0; mt < TM; ++mt) sha[mt] = a_at((wm * TM + mt) * 32 + (lane & 31)) & 3;
#pragma unroll
    for (int nt = 0; nt < TN; ++nt) shb[nt] = w_at((wn * TN + nt) * 32 + (lane & 31)) & 3;
  }
  // fragments of slice ks of stage st into set ks % kSets
  auto frags = [&](int st, int ks) {
    const int8_t* base = sm + st * G::kStage + (slot0 ^ (ks * 32));
#pragma unroll
    for (int mt = 0; mt < TM; ++mt) fa[ks % kSets][mt] = *reinterpret_cast<const v4i*>(base + arow + mt * 32 * BK);
#pragma unroll
    for (int nt = 0; nt < TN; ++nt) fb[ks % kSets][nt] = *reinterpret_cast<const v4i*>(base + brow + nt * 32 * BK);
    if constexpr (SHIFT) {
      // the word behind the fragment: the next chunk's first, or behind the last chunk the row's next word
      const bool last = ks == kSlices - 1;
      const int chunk = 2 * ks + kh + 1, slot = (chunk ^ swizzle(lane & 31)) * 16;
      const int8_t* stage = sm + st * G::kStage;
#pragma unroll
      for (int mt = 0; mt < TM; ++mt) {
        const int in = arow + mt * 32 * BK + slot, behind = G::kRows * BK + (wm * TM * 32 + mt * 32 + (lane & 31)) * 4;
        na[ks % kSets][mt] = *reinterpret_cast<const uint32_t*>(stage + (last && kh ? behind : in));
      }
#pragma unroll
      for (int nt = 0; nt < TN; ++nt) {
        const int in = brow + nt * 32 * BK + slot, behind = G::kRows * BK + (G::kBM + wn * TN * 32 + nt * 32 + (lane & 31)) * 4;
        nb[ks % kSets][nt] = *reinterpret_cast<const uint32_t*>(stage + (last && kh ? behind : in));
      }
    }
  };

  constexpr int kFirst = AHEAD == 1 ? NS : NS - 1;  // steps issued before the loop
  if (!tail) issue(0, 0);
#pragma unroll
  for (int d = 1; d < kFirst; ++d) issue(d, d);
  if (tail) {
    uint4 va[G::kNA], vw[G::kNB];
    uint32_t xw[G::kNX + 1];
#pragma unroll
    for (int i = 0; i < G::kNX; ++i)
      xw[i] = word_behind<BK>((xrow[i] < G::kBM ? abase : wbase) + (xoff[i] - BK + (xsh[i] ? 0 : 4)), full, p.K + xsh[i]);
    if (!SHIFT || p.K >= 16) {
#pragma unroll
      for (int i = 0; i < G::kNA; ++i) va[i] = load16(abase + aoff[i], full * BK + achk[i], p.K + atail[i]);
#pragma unroll
      for (int i = 0; i < G::kNB; ++i) vw[i] = load16(wbase + woff[i], full * BK + wchk[i], p.K + wtail[i]);
    } else {
#pragma unroll
      for (int i = 0; i < G::kNA; ++i) va[i] = load16_short(abase + aoff[i], achk[i], p.K + atail[i]);
#pragma unroll
      for (int i = 0; i < G::kNB; ++i) vw[i] = load16_short(wbase + woff[i], wchk[i], p.K + wtail[i]);
    }
#pragma unroll
    for (int i = 0; i < G::kNA; ++i) *reinterpret_cast<uint4*>(dst_a + i * 1024 + lane * 16) = va[i];
#pragma unroll
    for (int i = 0; i < G::kNB; ++i) *reinterpret_cast<uint4*>(dst_w + i * 1024 + lane * 16) = vw[i];
#pragma unroll
    for (int i = 0; i < G::kNX; ++i)
      *reinterpret_cast<uint32_t*>(sm + G::kRows * BK + (xrow[i] + lane) * 4) = xw[i];
  }
  wait_vm_lds<(kFirst - 1) * kLd>();
  __builtin_amdgcn_s_barrier();
  fence();
#pragma unroll
  for (int d = 0; d < AHEAD; ++d) frags(0, d);
  int st = 0;
  constexpr int kMf = TM * TN, kDs = TM + TN;
  for (int s = 0; s < nsteps; ++s) {
    const int nx = st + 1 == NS ? 0 : st + 1;
#pragma unroll
    for (int ks = 0; ks < kSlices; ++ks) {
      const bool cross = ks == kSlices - AHEAD;  // the next fragments are the next step's first
      if (cross) {
        if constexpr (AHEAD == 1) {
          // every wave has the last fragments of stage st in registers, and step s + 1 has landed
          wait_vm_lds<(NS - 2) * kLd>();
        } else {
          // step s + 1 has landed, and every wave has used all of step s - 1
          wait_vm<(NS - 3) * kLd>();
        }
        __builtin_amdgcn_s_barrier();
        fence();
      }
      frags(ks + AHEAD < kSlices ? st : nx, (ks + AHEAD) % kSlices);
      if (cross) {
        if constexpr (AHEAD == 1) issue(s + NS, st);
        else issue(s + NS - 1, st == 0 ? NS - 1 : st - 1);
      }
      if constexpr (SHIFT) {
#pragma unroll
        for (int mt = 0; mt < TM; ++mt) fa[ks % kSets][mt] = shifted(fa[ks % kSets][mt], na[ks % kSets][mt], sha[mt]);
#pragma unroll
        for (int nt = 0; nt < TN; ++nt) fb[ks % kSets][nt] = shifted(fb[ks % kSets][nt], nb[ks % kSets][nt], shb[nt]);
      }
#pragma unroll
      for (int mt = 0; mt < TM; ++mt)
#pragma unroll
        for (int nt = 0; nt < TN; ++nt)
          acc[mt][nt] = __builtin_amdgcn_mfma_i32_32x32x32_i8(fb[ks % kSets][nt], fa[ks % kSets][mt], acc[mt][nt], 0, 0, 0);
      // issue order: a product, two fragment reads, ... (after the barrier: then a product, a load, ...)
#pragma unroll
      for (int i = 0; i < kDs / 2; ++i) {
        __builtin_amdgcn_sched_group_barrier(0x8, 1, 0);
        __builtin_amdgcn_sched_group_barrier(0x100, SHIFT ? 4 : 2, 0);
      }
      if (cross) {
#pragma unroll
        for (int i = 0; i < kLd; ++i) {
          __builtin_amdgcn_sched_group_barrier(0x8, 1, 0);
          __builtin_amdgcn_sched_group_barrier(0x10, 1, 0);
        }
      }
      __builtin_amdgcn_sched_group_barrier(0x8, kMf, 0);
      __builtin_amdgcn_sched_barrier(0);
    }
    st = nx;
  }
  const int64_t mw = m0 + wm * TM * 32, nw = n0 + wn * TN * 32;
  s_sw += wn * TN * 32;
  s_bias += wn * TN * 32;
  bool all_tame = tame(s_sw[lane % (TN * 32)]);
#pragma unroll
  for (int mt = 0; mt < TM; ++mt) all_tame &= tame(sa[mt]);
  const bool wide = __any(!all_tame);
  wait_vm_lds<0>();  // no direct load outlives the stages it writes
  __syncthreads();   // every wave is done with them: they become the waves' output buffers
  const auto out = [&](auto w, auto t) {
    epilogue<decltype(w)::value, TM, TN, G::kBM == 256, decltype(t)>(p, sm, s_sw, s_bias, acc, sa, mw, nw, wave, lane);
  };
  if (__builtin_expect(wide, 0)) {
    if (p.yf16) out(std::true_type(), __half());
    else out(std::true_type(), float());
  } else {
    if (p.yf16) out(std::false_type(), __half());
    else out(std::false_type(), float());
  }
}

// ------------------------------------------------------------------------------------------------
// Tiles of (32 TM) x (32 TN) with K split over the W waves of a workgroup: wave k takes the units
// k, k + W, ... of BK bytes, each through NS LDS stages of its own that it fills and reads alone, so
// no barrier is needed until the waves' integer sums are joined (exactly, in any order) in LDS.
// ROWS: token rows that are loaded (a multiple of 1024 / BK; tokens past M up to ROWS read the last
// row, those past ROWS are whatever the LDS held: their sums are not stored). SHIFT: as in the shared tiles.
template <int TM, int TN, int BK, int W, int ROWS, int NS, bool SHIFT>
struct Split {
  static constexpr int kBM = TM * 32, kBN = TN * 32, kRpl = 1024 / BK;  // rows per load instruction
  static constexpr int kNA = ROWS / kRpl, kNB = kBN / kRpl;
  static constexpr int kNX = SHIFT ? 2 : 0;  // loads of the next words of 64 rows, half of them twice
  static constexpr int kStage = (kBM + kBN) * BK + kNX * 256, kRow = kBN + 4;
  static constexpr int kMain = NS * W * kStage, kEnd = W * kBM * kRow * 4;
  static constexpr int kLds = kMain > kEnd ? kMain : kEnd;
};

template <int TM, int TN, int BK, int W, int ROWS, int NS, bool SHIFT>
__global__ __launch_bounds__(W * 64, 2) void k_gemm_w8a8_split(GemmParams p) {
  using G = Split<TM, TN, BK, W, ROWS, NS, SHIFT>;
  constexpr int BM = G::kBM, BN = G::kBN, kSlots = BK / 16, kLd = G::kNA + G::kNB + G::kNX;
  static_assert(!SHIFT || (TM == 1 && TN == 1), "a lane's next words are of one row of each operand");
  __shared__ __align__(1024) int8_t sm[G::kLds];
  const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6), kh = lane >> 5;
  const int64_t nm = (p.M + BM - 1) / BM, nn = (p.N + BN - 1) / BN;
  const int64_t id = (int64_t)(blockIdx.x % 8) * (gridDim.x / 8) + blockIdx.x / 8;
  if (id >= nm * nn) return;  // grid padding (the whole workgroup)
  const int64_t m0 = id % nm * BM, n0 = id / nm * BN;
  const int8_t* abase = p.a + m0 * p.as;
  const int8_t* wbase = p.w + n0 * p.ws;
  const int apre = SHIFT ? (int)((uintptr_t)abase & 3) : 0, wpre = SHIFT ? (int)((uintptr_t)wbase & 3) : 0;
  abase -= apre;
  wbase -= wpre;
  constexpr int kWord = SHIFT ? ~3 : ~0;
  const int alast = (int)min(p.M - 1 - m0, (int64_t)BM), wlast = (int)min(p.N - 1 - n0, (int64_t)BN);
  const int as = (int)p.as, ws = (int)p.ws;
  const auto a_at = [&](int row) { return min(row, alast) * as + apre; };
  const auto w_at = [&](int row) { return min(row, wlast) * ws + wpre; };
  const int lrow = lane / kSlots;
  // load i: rows i kRpl ..., lane l at row l / kSlots, slot l % kSlots; byte offset of its chunk
  int aoff[G::kNA], woff[G::kNB], achk[G::kNA], wchk[G::kNB];
  uint32_t atail[G::kNA], wtail[G::kNB];  // codes before the row's first
#pragma unroll
  for (int i = 0; i < G::kNA; ++i) {
    const int row = i * G::kRpl + lrow;
    achk[i] = ((lane % kSlots) ^ swizzle(row)) * 16;
    aoff[i] = a_at(row) & kWord;
    atail[i] = a_at(row) & ~kWord;
  }
#pragma unroll
  for (int i = 0; i < G::kNB; ++i) {
    const int row = i * G::kRpl + lrow;
    wchk[i] = ((lane % kSlots) ^ swizzle(row)) * 16;
    woff[i] = w_at(row) & kWord;
    wtail[i] = w_at(row) & ~kWord;
  }
  // SHIFT: the lane's rows' codes before the first, and where the words behind a step lie
  const int ax = a_at(lane & 31), wx = w_at(lane & 31);
  const uint32_t sha = ax & 3, shb = wx & 3;
  const int axoff = (ax & ~3) + BK - (sha ? 0 : 4), wxoff = (wx & ~3) + BK - (shb ? 0 : 4);
  int8_t* mine = sm + wave * NS * G::kStage;
  const int full = (int)(p.K / BK);

  v16i acc[TM][TN];
#pragma unroll
  for (int mt = 0; mt < TM; ++mt)
#pragma unroll
    for (int nt = 0; nt < TN; ++nt) acc[mt][nt] = v16i{};
  auto products = [&](int st) {
    const int8_t* base = mine + st * G::kStage;
    v4i fa[BK / 32][TM], fb[BK / 32][TN];
#pragma unroll
    for (int ks = 0; ks < BK / 32; ++ks) {
      const int slot = ((2 * ks + kh) ^ swizzle(lane & 31)) * 16;
#pragma unroll
      for (int mt = 0; mt < TM; ++mt) fa[ks][mt] = *reinterpret_cast<const v4i*>(base + (mt * 32 + (lane & 31)) * BK + slot);
#pragma unroll
      for (int nt = 0; nt < TN; ++nt) fb[ks][nt] = *reinterpret_cast<const v4i*>(base + (BM + nt * 32 + (lane & 31)) * BK + slot);
    }
#pragma unroll
    for (int ks = 0; ks < BK / 32; ++ks)
      if constexpr (SHIFT) {
        const int slot = ((2 * ks + kh + 1) ^ swizzle(lane & 31)) * 16, row = lane & 31;
        const bool behind = ks == BK / 32 - 1 && kh;
        const int8_t* words = base + (BM + BN) * BK;
        fa[ks][0] = shifted(fa[ks][0], *reinterpret_cast<const uint32_t*>(behind ? words + row * 4 : base + row * BK + slot), sha);
        fb[ks][0] = shifted(fb[ks][0], *reinterpret_cast<const uint32_t*>(behind ? words + 256 + row * 4 : base + (BM + row) * BK + slot), shb);
      }
#pragma unroll
    for (int ks = 0; ks < BK / 32; ++ks)
#pragma unroll
      for (int mt = 0; mt < TM; ++mt)
#pragma unroll
        for (int nt = 0; nt < TN; ++nt)
          acc[mt][nt] = __builtin_amdgcn_mfma_i32_32x32x32_i8(fb[ks][nt], fa[ks][mt], acc[mt][nt], 0, 0, 0);
  };
  // a unit through registers, codes at or past K as 0
  auto to_lds = [&](const uint4 (&va)[G::kNA], const uint4 (&vw)[G::kNB]) {
#pragma unroll
    for (int i = 0; i < G::kNA; ++i) *reinterpret_cast<uint4*>(mine + i * 1024 + lane * 16) = va[i];
#pragma unroll
    for (int i = 0; i < G::kNB; ++i) *reinterpret_cast<uint4*>(mine + BM * BK + i * 1024 + lane * 16) = vw[i];
    wait_vm_lds<63>();
  };

  const __amdgpu_buffer_rsrc_t ra = rsrc_of(abase), rw = rsrc_of(wbase);
  // past the last unit the last one again, so that the waits stay exact
  auto issue = [&](int u, int st) {
    const int koff = min(u, full - 1) * BK;
#pragma unroll
    for (int i = 0; i < G::kNA; ++i) load_lds(ra, mine + st * G::kStage + i * 1024, aoff[i] + achk[i], koff);
#pragma unroll
    for (int i = 0; i < G::kNB; ++i) load_lds(rw, mine + st * G::kStage + BM * BK + i * 1024, woff[i] + wchk[i], koff);
    if constexpr (SHIFT) {
      load_lds_word(ra, mine + st * G::kStage + (BM + BN) * BK, axoff, koff);
      load_lds_word(rw, mine + st * G::kStage + (BM + BN) * BK + 256, wxoff, koff);
    }
  };
  if (wave < full) {
#pragma unroll
    for (int d = 0; d < NS; ++d) issue(wave + d * W, d);
    int st = 0;
    for (int u = wave; u < full; u += W) {
      wait_vm_lds<(NS - 1) * kLd>();
      products(st);
      wait_vm_lds<63>();  // the stage's fragments are in registers
      issue(u + NS * W, st);
      st = st + 1 == NS ? 0 : st + 1;
    }
    wait_vm_lds<0>();
  }
  // the last K % BK codes
  if (p.K % BK != 0 && wave == full % W) {
    uint4 va[G::kNA], vw[G::kNB];
    uint32_t xa = 0u, xw = 0u;
    if constexpr (SHIFT) {
      xa = word_behind<BK>(abase + (ax & ~3), full, p.K + sha);
      xw = word_behind<BK>(wbase + (wx & ~3), full, p.K + shb);
    }
#pragma unroll
    for (int i = 0; i < G::kNA; ++i) va[i] = load16(abase + aoff[i], full * BK + achk[i], p.K + atail[i]);
#pragma unroll
    for (int i = 0; i < G::kNB; ++i) vw[i] = load16(wbase + woff[i], full * BK + wchk[i], p.K + wtail[i]);
    if constexpr (SHIFT) {
      *reinterpret_cast<uint32_t*>(mine + (BM + BN) * BK + lane * 4) = xa;
      *reinterpret_cast<uint32_t*>(mine + (BM + BN) * BK + 256 + lane * 4) = xw;
    }
    to_lds(va, vw);
    products(0);
  }

  __syncthreads();
  int* red = reinterpret_cast<int*>(sm);  // [wave][row][column]
#pragma unroll
  for (int mt = 0; mt < TM; ++mt)
#pragma unroll
    for (int nt = 0; nt < TN; ++nt)
#pragma unroll
      for (int j = 0; j < 4; ++j)
        *reinterpret_cast<v4i*>(red + (wave * BM + mt * 32 + (lane & 31)) * G::kRow + nt * 32 + 8 * j + 4 * kh) =
            v4i{acc[mt][nt][4 * j], acc[mt][nt][4 * j + 1], acc[mt][nt][4 * j + 2], acc[mt][nt][4 * j + 3]};
  __syncthreads();
  for (int i = threadIdx.x; i < BM * BN / 4; i += W * 64) {
    const int row = i / (BN / 4), col = i % (BN / 4) * 4;
    const int64_t m = m0 + row;
    if (m >= p.M) continue;
    v4i v = *reinterpret_cast<const v4i*>(red + row * G::kRow + col);
#pragma unroll
    for (int q = 1; q < W; ++q) v += *reinterpret_cast<const v4i*>(red + (q * BM + row) * G::kRow + col);
    const float sa = valid_or_zero(p.a_scales[p.per_row ? m : 0]);
    float sw[4], bias[4], o[4];
    bool all_tame = tame(sa);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int64_t n = min(n0 + col + k, p.N - 1);
      sw[k] = valid_or_zero(p.w_scales[n]);
      bias[k] = p.bias ? p.bias[n] : 0.0f;
      all_tame &= tame(sw[k]);
      o[k] = scaled(sa, sw[k], v[k], bias[k]);
    }
    if (!all_tame) {
#pragma unroll
      for (int k = 0; k < 4; ++k) o[k] = scaled_wide(sa, sw[k], v[k], bias[k]);
    }
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (n0 + col + k < p.N) put(p, m, n0 + col + k, o[k]);
  }
}

// ------------------------------------------------------------------------------------------------
unsigned grid_of(const GemmParams& p, int bm, int bn) { return (unsigned)(cdiv(cdiv(p.M, bm) * cdiv(p.N, bn), 8) * 8); }

template <bool SHIFT>
void launch_tile(Form form, const GemmParams& p, hipStream_t stream) {
  switch (form) {
    case TILE256: k_gemm_w8a8_tile<2, 4, 4, 2, 2, 128, 1, SHIFT><<<grid_of(p, 256, 256), 512, 0, stream>>>(p); break;
    case TILE256X128: k_gemm_w8a8_tile<4, 2, 2, 2, 3, 128, 1, SHIFT><<<grid_of(p, 256, 128), 512, 0, stream>>>(p); break;
    case TILE128: k_gemm_w8a8_tile<2, 2, 2, 2, 3, 128, 1, SHIFT><<<grid_of(p, 128, 128), 256, 0, stream>>>(p); break;
    case TILE128X64: k_gemm_w8a8_tile<2, 2, 2, 1, 3, 128, 1, SHIFT><<<grid_of(p, 128, 64), 256, 0, stream>>>(p); break;
    case TILE64: k_gemm_w8a8_tile<2, 2, 1, 1, 3, 128, 1, SHIFT><<<grid_of(p, 64, 64), 256, 0, stream>>>(p); break;
    default:
      if constexpr (!SHIFT) k_gemm_w8a8_tile<2, 2, 1, 1, 6, 128, 3, false><<<grid_of(p, 64, 64), 256, 0, stream>>>(p);
  }
}

template <int ROWS, bool SHIFT>
void launch_split(const GemmParams& p, hipStream_t stream) {
  k_gemm_w8a8_split<1, 1, 128, 4, ROWS, 2, SHIFT><<<grid_of(p, 32, 32), 256, 0, stream>>>(p);
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
  const int64_t lim = (int64_t)1 << 40;
  if (a->a_stride > lim || a->w_stride > lim || a->y_stride > lim || M > (1 << 27) || N > (1 << 27))
    return fail(QSSM_ERR_UNSUPPORTED, "M or N above 2^27 or a stride above 2^40");
  if (a->y_stride > ((int64_t)1 << 58) / std::max<int64_t>(M, 1))  // row offsets in bytes stay inside 64 bits
    return fail(QSSM_ERR_UNSUPPORTED, "M * y_stride above 2^58");
  if (M == 0 || N == 0) return QSSM_OK;
  if (!a->a_scales || !a->w_scales || !a->y || (K > 0 && (!a->a || !a->w)))
    return fail(QSSM_ERR_INVALID_ARG, "null required pointer");
  if (((uintptr_t)a->y) % (a->y_dtype == QSSM_F16 ? 2 : 4) != 0)
    return fail(QSSM_ERR_INVALID_ARG, "y is not aligned to its type");
  if (((uintptr_t)a->a_scales | (uintptr_t)a->w_scales | (uintptr_t)a->bias) % 4 != 0)
    return fail(QSSM_ERR_INVALID_ARG, "a_scales, w_scales or bias is not aligned to its type");
  // 32-bit offsets inside a tile
  if (std::max(a->a_stride, a->w_stride) > (1 << 22))
    return fail(QSSM_ERR_UNSUPPORTED, "a_stride or w_stride above 2^22");
  // a grid holds fewer than 2^32 threads, 512 a workgroup
  if (cdiv(M, 256) * cdiv(N, 128) >= kMaxTiles) return fail(QSSM_ERR_UNSUPPORTED, "M * N too large");
  const Span y{a->y, M, a->y_stride * (a->y_dtype == QSSM_F16 ? 2 : 4), N * (a->y_dtype == QSSM_F16 ? 2 : 4)};
  if (overlap(y, Span{a->a, M, a->a_stride, K}) || overlap(y, Span{a->w, N, a->w_stride, K}) || overlap(y, flat(a->bias, N * 4)) ||
      overlap(y, flat(a->a_scales, a->a_per_row ? M * 4 : 4)) || overlap(y, flat(a->w_scales, N * 4)))
    return fail(QSSM_ERR_INVALID_ARG, "y overlaps an input");
  const GemmParams p{M, N, K, a->a_per_row != 0, a->y_dtype == QSSM_F16, a->a, a->a_stride, a->a_scales,
                     a->w, a->w_stride, a->w_scales, a->bias, a->y, a->y_stride};
  const bool direct = ((uintptr_t)a->a | (uintptr_t)a->w | (uintptr_t)a->a_stride | (uintptr_t)a->w_stride) % 4 == 0;
  const auto [form, shift] = choose_form(M, N, K, p.yf16, direct);
  if (form == SPLIT32) {
    // up to 16 tokens load only 16 of a tile's 32 rows (8 tokens x 18560 x 4096: 18.9 us, 19.9 with all)
    if (M <= 16) shift ? launch_split<16, true>(p, stream) : launch_split<16, false>(p, stream);
    else shift ? launch_split<32, true>(p, stream) : launch_split<32, false>(p, stream);
  } else {
    shift ? launch_tile<true>(form, p, stream) : launch_tile<false>(form, p, stream);
  }
  return launch_status("gemm_w8a8");
}
