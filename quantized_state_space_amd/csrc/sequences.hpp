// Packed sequences and their state cache: what the causal convolution and the selective scan share.
#pragma once

#include "common.hpp"

namespace qssm {

constexpr int64_t kMaxSeqTokens = ((int64_t)1 << 31) - 64, kMaxSeqs = 1 << 24, kMaxSeqDim = 1 << 24;

struct Seqs {
  const int32_t* offsets;  // null: nseq sequences of `each` rows
  const int32_t* slot_of;  // null: slot i
  const uint8_t* has;      // null: 1
  int32_t tokens, nseq, each;
  int64_t slots;
};

// Sequence i's first row and the row behind its last, inside 0 .. tokens whatever the offsets hold.
__device__ __forceinline__ int seq_begin(const Seqs& s, int i) {
  return s.offsets ? min(max(s.offsets[i], 0), s.tokens) : i * s.each;
}

__device__ __forceinline__ int seq_end(const Seqs& s, int i, int begin) {
  return s.offsets ? max(min(s.offsets[i + 1], s.tokens), begin) : begin + s.each;
}

// Sequence i's slot, -1 without one.
__device__ __forceinline__ int64_t seq_slot(const Seqs& s, int i) {
  const int64_t k = s.slot_of ? (int64_t)s.slot_of[i] : (int64_t)i;
  return k >= 0 && k < s.slots ? k : -1;
}

// The largest i in 0 .. n - 1 with key(i) <= v, 0 if there is none, for keys that do not decrease: 64 of them
// at a time, one a lane, so that up to 64 sequences cost one load and up to 4096 two. Whole waves call it.
template <typename Key>
__device__ __forceinline__ int last_not_above(int n, int64_t v, Key key) {
  const int lane = threadIdx.x & 63;
  int lo = 0;
  while (n > 1) {
    const int step = (n + 63) / 64, at = lane * step;
    const bool in = at < n && key(lo + (at < n ? at : 0)) <= v;
    const int k = max((int)__popcll(__ballot(in)) - 1, 0) * step;  // (__popcll is unsigned)
    lo += k;
    n = min(step, n - k);
  }
  return uniform(lo);
}

// ---------------------------------------------------------------------------------------------
// Host: the checks of what the sequences need.
inline int64_t type_size(int32_t t) { return t == QSSM_F16 ? 2 : t == QSSM_I8 ? 1 : 4; }

inline qssm_status check_seqs(int64_t tokens, int64_t dim, int64_t nseq, const void* offsets, const void* state,
                              const void* state_out, int64_t slots, const void* slot_of) {
  if (tokens < 0 || dim < 0 || nseq < 0 || slots < 0) return fail(QSSM_ERR_INVALID_ARG, "negative extent");
  if (tokens > kMaxSeqTokens || dim > kMaxSeqDim || nseq > kMaxSeqs)
    return fail(QSSM_ERR_UNSUPPORTED, "tokens above 2^31 - 64, or dim or nseq above 2^24");
  if (!offsets && (nseq == 0 ? tokens != 0 : tokens % nseq != 0))
    return fail(QSSM_ERR_INVALID_ARG, "tokens is not a multiple of nseq (and there are no seq_offsets)");
  if ((uintptr_t)offsets % 4 != 0 || (uintptr_t)slot_of % 4 != 0)
    return fail(QSSM_ERR_INVALID_ARG, "seq_offsets or state_slots is not aligned to its type");
  if (state || state_out) {
    if (slots > ((int64_t)1 << 40)) return fail(QSSM_ERR_UNSUPPORTED, "slots above 2^40");
    if (!slot_of && slots < nseq) return fail(QSSM_ERR_INVALID_ARG, "fewer slots than sequences (and no state_slots)");
  }
  return QSSM_OK;
}

// Rows of a 2-D tensor of `cols` elements of `size` bytes.
inline qssm_status check_rows(const char* name, const void* p, int64_t rows, int64_t cols, int64_t stride, int64_t size) {
  if (!p) return QSSM_OK;
  if (stride < cols) return fail(QSSM_ERR_INVALID_ARG, "%s_stride is smaller than the row", name);
  if (stride > ((int64_t)1 << 40) || stride > ((int64_t)1 << 58) / std::max<int64_t>(rows, 1))
    return fail(QSSM_ERR_UNSUPPORTED, "%s_stride above 2^40, or rows * stride above 2^58", name);
  if ((uintptr_t)p % size != 0) return fail(QSSM_ERR_INVALID_ARG, "%s is not aligned to its type", name);
  return QSSM_OK;
}

inline Seqs make_seqs(int64_t tokens, int64_t nseq, const int32_t* offsets, const int32_t* slot_of, const uint8_t* has,
                      int64_t slots) {
  return Seqs{offsets, slot_of, has, (int32_t)tokens, (int32_t)nseq, (int32_t)(nseq > 0 ? tokens / nseq : 0), slots};
}

}  // namespace qssm
