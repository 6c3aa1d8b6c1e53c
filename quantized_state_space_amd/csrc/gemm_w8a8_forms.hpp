// The forms of the W8A8 linear layer and the choice among them (host only, no HIP: tests build it alone).
#pragma once

#include <stdint.h>

#include <algorithm>
#include <cmath>

namespace qssm {

// The form for a shape, by estimated time (us): a tile costs tile + step * (steps of 64 codes of K) of
// its CU when it shares it, tile_alone + step_alone * steps when the last round leaves it alone there;
// the whole at least the bytes at 4.3 TB/s. The constants follow a fit (16 % rms) to 30 shapes of 1 .. 16384
// tokens, N = 1024 .. 18560 and K = 128 .. 8192 in every form; they named the fastest form at 27 of them
// and one within 3 to 14 % of it at the others. Measured, e.g. (256x256 / 256x128 / 128x128 / 128x64 /
// 64x64 / split 32x32 / deep 64x64; weights in the last-level cache):
//   64 x 4096 x 8192      71 / 38 / 29 / 20 / 17 / 9.1 / 15     256 x 4096 x 8192   73 / 39 / 30 / 22 / 18 / 24 / 15.7
//   1000 x 1536 x 768     13 / 8.4 / 7.5 / 5.8 / 5.5 / 11 / 7.7 256 x 18560 x 4096  41 / 25 / 36 / 32 / 33 / 60 / 41
//   1024 x 4096 x 4096    40 / 24 / 21 / 23 / 29 / 57 / 34      4096 x 4096 x 4096  58 / 64 / 79 / 90 / 111 / 283 / 131
// Not covered: few tokens and weights of more than ~75 MB. There several forms lie below the line of the bytes,
// tie, and the first in the order below is taken, which is up to a third slower than the fastest:
//   1 x 18560 x 8192      72 / 40 / 29 (taken) / 29 / 24 / 24 / 33   64 x 50288 x 4096   46 (taken) / 50 / 39 / 39 / 36 / 46 / 42
//   1 x 50288 x 4096      43 (taken) / 48 / 38 / 36 / 35 / 33 / 40   1 x 16384 x 8192    72 / 38 / 29 / 22 (taken) / 21 / 20 / 21
enum Form { TILE256, TILE256X128, TILE128, TILE128X64, TILE64, SPLIT32, TILE64DEEP, FORMS };
struct FormCost {
  int bm, bn, per_cu;
  double tile, step, tile_alone, step_alone;
};
constexpr FormCost kFormCost[FORMS] = {{256, 256, 1, 0.0, 0.68, 6.0, 0.591},    {256, 128, 1, 4.31, 0.321, 4.31, 0.321},
                                       {128, 128, 1, 3.93, 0.231, 3.93, 0.231}, {128, 64, 2, 1.48, 0.164, 2.56, 0.156},
                                       {64, 64, 3, 0.87, 0.104, 1.65, 0.111},   {32, 32, 2, 1.26, 0.048, 1.26, 0.048},
                                       {64, 64, 1, 1.0, 0.132, 1.0, 0.101}};

constexpr int64_t kMaxTiles = ((int64_t)1 << 23) - 8;

// The cheapest of the first n forms.
inline Form cheapest_form(int64_t M, int64_t N, int64_t K, bool yf16, int n) {
  constexpr double kCus = 256.0;
  const auto pieces = [](int64_t v, int64_t by) { return (double)((v + by - 1) / by); };
  const double steps = pieces(K, 64);
  const double bytes = ((double)M + (double)N) * (double)K + (yf16 ? 2.0 : 4.0) * (double)M * (double)N;
  int best = -1;
  double least = 0.0;
  for (int f = 0; f < n; ++f) {
    const FormCost& c = kFormCost[f];
    const double tiles = pieces(M, c.bm) * pieces(N, c.bn), slots = kCus * c.per_cu;
    if (tiles >= (double)kMaxTiles) continue;
    const double busy = c.tile + c.step * steps, alone = c.tile_alone + c.step_alone * steps;
    const double rounds = std::ceil(tiles / slots) - 1.0, on_cu = std::ceil((tiles - rounds * slots) / kCus);
    const double last = on_cu <= 1.0 ? alone : std::max(alone, busy * on_cu);
    const double t = std::max(rounds * c.per_cu * busy + last, bytes / 4.3e6);
    if (best < 0 || t < least) {
      least = t;
      best = f;
    }
  }
  return (Form)best;
}

struct FormChoice {
  Form form;
  bool shift;  // the form for rows at any address
};

// direct: a, w and their strides are multiples of 4 bytes, as direct loads need. Other rows, and in the tiles a K
// without a full step, take the shifted forms: the fastest at the same estimates or within 6 % of it in 12 shapes
// of 1 .. 16384 tokens. The split form needs K >= 16 (1 x 1000 x 64: 3.8 us, a shifted tile 4.5).
inline FormChoice choose_form(int64_t M, int64_t N, int64_t K, bool yf16, bool direct) {
  const Form f = cheapest_form(M, N, K, yf16, direct && K >= 128 ? FORMS : K >= 16 ? TILE64DEEP : SPLIT32);
  return {f, !direct || (K < 128 && f != SPLIT32)};
}

}  // namespace qssm
