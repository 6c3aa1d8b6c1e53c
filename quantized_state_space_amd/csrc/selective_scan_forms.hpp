// How the selective scan cuts its sequences and where it keeps their pieces' ends (no HIP: tests build it alone).
#pragma once

#include <stdint.h>

#include <algorithm>

namespace qssm_sscan {

constexpr int64_t kLeastPiece = 64, kMostPiece = 256, kPieceStep = 32;

// Rows of a piece. A cut costs nearly twice the work, and pays where whole sequences leave SIMDs (1024 of them) without a
// wave or wait for the longest one: sequences of one length that give nearly all of them a wave run whole (16 of
// 1024 rows, 4096 channels: 298 us, 431 in pieces of 256; 8 of 1024, 1536 channels, three quarters of the SIMDs: 120,
// and 103 in pieces of 128); others run in pieces that give about 6 waves a SIMD, of 64 to 256 rows (1 x 8192
// rows, 1536 channels, pieces of 64 / 128 / 256 / 512: 147 / 123 / 118 / 149 us, whole 900; 24 sequences of very different
// lengths, 16384 rows, 4096 channels, 128 / 256 / 384 / 512: 466 / 433 / 438 / 450, whole 708; 100 of them, 1536 channels:
// 191 / 198 / 230 / 272, 220). The six waves are a compromise over these: the one prompt runs in pieces of 128 and the hundred
// sequences in 256, each 4 % from its best, and the registers hold four waves of 16 states a SIMD, which the rule does not count.
// waves: of one piece, over its channels; packed: with offsets.
inline int64_t piece_rows(int64_t tokens, int64_t nseq, int64_t waves, bool packed) {
  const int64_t whole = std::max<int64_t>(tokens, 1);
  if (!packed && nseq * waves >= 900) return whole;
  return std::min<int64_t>(whole, std::clamp<int64_t>((whole * waves / 6144 + 16) / kPieceStep * kPieceStep, kLeastPiece, kMostPiece));
}

// Whether a sequence may have more than a piece's rows.
inline bool is_cut(int64_t tokens, int64_t nseq, int64_t piece, bool packed) {
  return piece < (packed ? tokens : tokens / std::max<int64_t>(nseq, 1));
}

// The workspace's slots, one for each piece of a sequence of more than `piece` rows: the first one of sequence i, with f =
// (its first row) / piece. Such a sequence of len rows ends in f' > f and has ceil(len / piece) <= f' - f + 1 pieces, and
// i and f both grow by 1 or more up to the next one, so that their least does: no slots overlap, and all lie below
// carry_slots(), the latter also where offsets are out of order.
constexpr int first_slot(int i, int f) { return f + (i < f ? i : f); }

inline int64_t carry_slots(int64_t tokens, int64_t nseq, int64_t piece) { return tokens / piece + std::min(nseq, tokens / piece); }

// The most that carry_slots() gives for up to `tokens` rows in any number of sequences: for each length of a piece, at its
// largest number of rows.
inline int64_t most_slots(int64_t tokens, int64_t waves) {
  int64_t most = 0;
  for (int64_t p = kLeastPiece; p <= kMostPiece; p += kPieceStep) {
    const int64_t rows = p == kMostPiece ? tokens : std::min(tokens, ((p + kPieceStep - 16) * 6144 - 1) / waves);
    most = std::max(most, 2 * (rows / p));
  }
  return most;
}

// Single rows: four sequences a lane (of states 4 * npl <= 32) where that leaves a wave to every SIMD; blocks: workgroups of a sequence.
inline bool four_at_a_time(int64_t nseq, int64_t blocks, int npl) { return npl <= 8 && (nseq + 3) / 4 * blocks >= 256; }

}  // namespace qssm_sscan
