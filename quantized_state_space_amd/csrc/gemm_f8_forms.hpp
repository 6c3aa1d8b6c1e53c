// The forms of the block-scaled e4m3 linear layer and the choice among them (host only, no HIP: tests build it alone).
#pragma once

#include <stdint.h>

#include <algorithm>
#include <cmath>

namespace qssm_f8 {

// The tile form for a shape, by estimated time (us): a tile costs tile + step * (blocks of K) of its CU when it shares it,
// tile_alone + step_alone * blocks when the last round leaves it alone there; the whole at least the bytes at 4.3 TB/s.
// The constants follow a fit (10 to 27 % rms) to 30 shapes of 17 .. 16384 tokens, N = 200 .. 18560 and K = 200 .. 8192 in
// every form, of either type of y; the form that they name takes 1.3 % (fp16) and 2.1 % (fp32) more than the fastest
// in the mean. Measured, fp16 y, us (256x256 / 256x128 / 128x128 / 64x64 / 64x64 K2 / K4 / 32x32 K4 / K4 deep):
//   64 x 4096 x 8192   102 / 56 / 48 / 28 / 20 / 21 / 15 / 12     256 x 4096 x 8192   106 / 58 / 48 / 29 / 23 / 22 / 37 / 42
//   256 x 18560 x 4096  59 / 36 / 46 / 43 / 60 / 61 / 85 / 122    1024 x 4096 x 4096   59 / 34 / 31 / 39 / 46 / 47 / 74 / 103
//   777 x 1000 x 1536   31 / 18 / 16 / 9.4 / 8.3 / 8.8 / 12 / 18  4096 x 4096 x 4096   74 / 83 / 93 / 130 / 172 / 179 / 280 / 407
// 256x256 is for an fp16 y alone: with operands as fp16 (an fp32 y) its fragments leave the registers (4096 x 4096 x 4096:
// 188 us, 133 in 256x128).
enum Form { TILE256, TILE256X128, TILE128, TILE64, TILE64K2, TILE64K4, TILE32K4, TILE32K4DEEP, FORMS };
struct FormCost {
  int bm, bn, per_cu;
  double tile, step, tile_alone, step_alone;
};
constexpr FormCost kFormCost[2][FORMS] = {
    // fp32 y
    {{256, 256, 1, 0.7, 6.5, 13.5, 4.13},
     {256, 128, 1, 5.72, 1.865, 10.28, 1.34},
     {128, 128, 1, 1.92, 0.903, 9.67, 0.881},
     {64, 64, 3, 0.43, 0.373, 7.79, 0.455},
     {64, 64, 1, 3.68, 0.314, 6.38, 0.315},
     {64, 64, 1, 4.68, 0.295, 7.59, 0.28},
     {32, 32, 2, 2.02, 0.094, 6.96, 0.201},
     {32, 32, 1, 4.27, 0.115, 7.08, 0.161}},
    // fp16 y
    {{256, 256, 1, 1.0, 2.337, 12.97, 1.465},
     {256, 128, 1, 3.3, 1.104, 9.18, 0.779},
     {128, 128, 1, 1.27, 0.569, 8.72, 0.638},
     {64, 64, 3, 0.51, 0.209, 6.98, 0.36},
     {64, 64, 1, 2.85, 0.25, 7.04, 0.221},
     {64, 64, 1, 3.78, 0.238, 7.65, 0.21},
     {32, 32, 2, 1.77, 0.085, 7.3, 0.169},
     {32, 32, 1, 3.86, 0.089, 7.43, 0.111}}};

constexpr int64_t kMaxTiles = ((int64_t)1 << 23) - 8;  // a grid holds fewer than 2^32 threads, 512 a workgroup (1024: half)

inline Form choose_form(int64_t M, int64_t N, int64_t K, bool yf16) {
  constexpr double kCus = 256.0;
  const auto pieces = [](int64_t v, int64_t by) { return (double)((v + by - 1) / by); };
  const double steps = pieces(K, 128);
  const double bytes = ((double)M + (double)N) * (double)K + (yf16 ? 2.0 : 4.0) * (double)M * (double)N;
  int best = TILE256X128;
  double least = 0.0;
  for (int f = yf16 ? TILE256 : TILE256X128; f < FORMS; ++f) {
    const FormCost& c = kFormCost[yf16][f];
    const double tiles = pieces(M, c.bm) * pieces(N, c.bn), slots = kCus * c.per_cu;
    if (f > TILE256X128 && tiles >= (double)kMaxTiles / 2) continue;
    const double busy = c.tile + c.step * steps, alone = c.tile_alone + c.step_alone * steps;
    const double rounds = std::ceil(tiles / slots) - 1.0, on_cu = std::ceil((tiles - rounds * slots) / kCus);
    const double last = on_cu <= 1.0 ? alone : std::max(alone, busy * on_cu);
    const double t = std::max(rounds * c.per_cu * busy + last, bytes / 4.3e6);
    if (least == 0.0 || t < least) {
      least = t;
      best = f;
    }
  }
  return (Form)best;
}

}  // namespace qssm_f8
