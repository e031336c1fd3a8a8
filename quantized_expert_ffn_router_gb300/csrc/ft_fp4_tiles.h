// ft_fp4_tiles.h -- which tiles a product of 4-bit matrices takes: a rule on its
// sizes and the number of SMs, plain C++ that the host's tests compile too.
#pragma once

#include <stdint.h>

#include <algorithm>

namespace ft {

constexpr int kM = 128;     // weight rows of a tile (of each CTA of a pair)
constexpr int kStep = 256;  // values of K in a step: four products of 64
constexpr int kMaxWidth = 256;

struct Tiles {
  int pair;    // CTAs of a tile: 1 or 2
  int width;   // tokens of a tile
  int slices;  // of K, one a CTA of a cluster
};

inline int64_t tiles_of(int64_t T, int64_t N, int width, int pair) {
  return ((N - 1) / (kM * pair) + 1) * ((T - 1) / width + 1);
}

// Tiles and slices of K by what they take together (us, measured; what all of
// them take, 3.5 and the bytes from HBM, left out).  A step: issuing its copies
// and products, or the products themselves where they are wide.  After the last
// step the tile's sums are drained and written, 0.7 for 64 tokens, under the
// next tile's steps where there are two accumulators.  A pair of CTAs meets
// first; slices meet before and after their sums are joined.  E.g. 2048 x 4096 x
// 4096: pairs of 256 tokens 18.6, alone 20.7, of 128 24.3; 777 x 2560 x 2560:
// alone of 128 7.7, of 64 10.2, pairs 8.9; 300 x 300 x 8192: 8 slices of 64 7.5,
// whole 13.2; 64 x 2560 x 2048: whole 6.5, 4 slices 7.1.
inline Tiles choose_tiles(int64_t T, int64_t N, int steps, int sms) {
  constexpr double kStepUs[2][4] = {{0.255, 0.285, 0.32, 0.365}, {0.255, 0.28, 0.29, 0.303}};
  Tiles least = {1, 0, 1};
  double best = 0;
  const auto consider = [&](int pair, int width, int slices) {
    const int64_t tiles = tiles_of(T, N, width, pair), places = sms / (pair * slices);
    if (places < 1 || (slices > 1 && (tiles > places || slices > steps))) return;
    const int64_t waves = (tiles + places - 1) / places;
    const double tokens = width / 64.0;
    const double run = (steps + slices - 1) / slices * kStepUs[pair - 1][width > 64 ? width / 64 - 1 : 0];
    const double drain = 0.7 * tokens, wait = std::max(width > 128 ? 0.6 : 0.0, drain - run);
    const double cost =
        (pair == 2 ? 1.1 : 0) + waves * run + drain + (waves - 1) * wait + (slices > 1 ? 1.1 + 1.1 * tokens : 0);
    if (best == 0 || cost < best) best = cost, least = {pair, width, slices};
  };
  for (int slices = 1; slices <= 8; slices *= 2) {
    if (T <= 64) {
      consider(1, static_cast<int>(T + 15) / 16 * 16, slices);
      continue;
    }
    for (int width = 64; width <= kMaxWidth; width += 64) {
      consider(1, width, slices);
      if (slices == 1) consider(2, width, 1);
    }
  }
  return least;
}

}  // namespace ft
