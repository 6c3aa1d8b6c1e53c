// How the causal convolution cuts its rows into strips (no HIP: tests build it alone).
#pragma once

#include <stdint.h>

namespace qssm_conv {

// Rows of a strip, over `cblocks` blocks of channels: as long as leaves 8 waves to a SIMD (1024 SIMDs), 8 to 64 rows (16384 rows, 8192
// channels, at most 32 / 64 / 128: 146 / 140 / 142 us; 2777 rows, 1543 channels, 4 / 8 waves: 12.2 / 11.7)
inline int64_t strip_rows(int64_t tokens, int64_t cblocks) {
  int64_t strip = 64;
  while (strip > 8 && (tokens + strip - 1) / strip * cblocks < 8192) strip /= 2;
  return strip;
}

}  // namespace qssm_conv
