// The choice of tiles for a matrix product of linear.cu: plain C++ without CUDA, so that it can be
// asked on any machine.
#pragma once

#include <algorithm>

namespace moe {

constexpr int kTileI = 128;  // rows of a CTA's tile

// Which kernel and tiles take a product: the least of an estimate in microseconds, fitted to
// measurements of 16 to 1024 rows at 2048 x 7168, 8192 x 2048, 1536 x 4096, 4096 x 1024 and
// 512 x 1000 (within 20 % of them, and its choice within 10 % of the best there; elsewhere up to 17 %
// were seen: 256 x 4096 x 4096 16.7 us where 64 columns take 14.3).
// A step of 64 k takes a CTA 0.155 us up to 64 columns, 0.225 for 128 (0.29 with one block of k a
// stage) and 0.34 for 256, or what all CTAs' bytes take at 18 TB/s; a pair's 256 x 256 x 64 takes
// 0.29 us. Starting, filling the pipeline and the last products take 2 us (pairs, with their end:
// 7), an epilogue 0.4 us and 0.05 us for 1000 elements (0.35 us where rows do not start on 16
// bytes; 7 us for a pair). Joining S partial tiles costs 1.4 us and what a CTA's sums take to the
// others at 22 GB/s.
// Clusters of 1, 2, 4 and 8 of these CTAs: 152, 76, 36 and 15 fit on the GPU at once.
constexpr double kPairStart = 7.0, kPairStep = 0.29;
struct TileChoice {
  int bn, splits;  // bn -1: the pair kernel
  double us;
};
inline TileChoice choose_tiles(int I, int J, int nk, bool b_mn, bool aligned, int num_sms) {
  const long long ti = (I + kTileI - 1) / kTileI;
  const long long t256 = ((long long)I + 255) / 256 * (((long long)J + 255) / 256);
  const long long pairs = num_sms / 2;
  TileChoice best{-1, 1, kPairStart + (aligned ? 0.0 : 7.0) +
                             (double)((t256 + pairs - 1) / pairs) * nk * kPairStep};
  const int rows = std::min(I, kTileI);
  for (int bn = b_mn ? 64 : 16; bn <= 256; bn *= 2) {
    if (bn < 64 && bn < J) continue;  // under 64 columns only for all of J
    const long long tiles = ti * ((J + bn - 1) / bn);
    const double bytes = (double)(rows + bn) * 128;
    for (int s = 1; s <= 8; s *= 2) {
      if (s > 1 && (nk < 2 * s || bn > 128)) break;  // 256 columns leave no room for the sums
      const long long fit = s == 1   ? num_sms
                            : s == 2 ? num_sms / 2
                            : s == 4 ? 36LL * num_sms / 152
                                     : 15LL * num_sms / 152;
      const double waves = (double)((tiles + fit - 1) / std::max(1LL, fit));
      const double busy = (double)(std::min(tiles, fit) * s);
      const double step = std::max(bn <= 64 ? 0.155 : bn == 256 ? 0.34 : s == 1 ? 0.225 : 0.29,
                                   bytes * busy / 18e6);
      const double join = (s == 1 ? 0.4 + (aligned ? rows * bn * 5e-5 : 0.0)
                                  : 1.4 + (double)rows * bn * 4 / 22e3) +
                          (aligned ? 0.0 : rows * bn * 3.5e-4 / s);
      const double us = 2.0 + waves * (step * ((nk + s - 1) / s) + join);
      if (us < best.us) best = TileChoice{bn, s, us};
    }
    if (bn >= J && bn >= 64) break;
  }
  return best;
}

}  // namespace moe
