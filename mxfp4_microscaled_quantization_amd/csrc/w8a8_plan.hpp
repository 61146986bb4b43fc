// Which kernel the 8-bit product takes for a shape (host only, no HIP): the tile, the parts of K, how
// the last round of the largest tile is cut, and whether rows off the cache lines take the shifted
// form.  gemm_int8.hip launches by it and sizes its workspace by it.
#pragma once

#include <stdint.h>

namespace mxq {

constexpr int kWin = 128;                    // K elements (bytes) per row per window
constexpr int kMaxSplits = 8;                // parts of K
constexpr int kFewTokens = 8;                // up to so many tokens the tiles are not used

// Choice of the tile, and of a split of K.  Every kernel gives the same sums, so this is
// about time alone.  A round of up to 256 tiles (one for each CU) takes fixed + per_window
// * windows us with the tile in question, kLaunch of it once; a further round takes `again`
// of the first (less than 1 where two workgroups fit a CU), or what dispatching 256 workgroups
// takes (4052 x 80 x 1491: 64 x 64 tiles 13.3 us, 32 x 32 28); a split of K adds the reduction
// and its traffic.  The constants are fits to times with cold operands, K = 5120 and 13824.
// So a small tile is taken until a larger one fills the CUs, and the largest past that:
//   512 x 5120 x 5120: 256 x 256 58 us, 128 x 256 40, 128 x 128 28, 64 x 128 40, 64 x 64 34
//   2048 x 5120 x 5120: 57, 78, 79, 99, 102;  128 x 5120 x 5120: 60, 43, 29, 22, 15.5
//   64 x 13824 x 5120: 64 x 32 27.5, 64 x 64 36, 64 x 64 in 3 parts of K 20.6
// off_lines: factor on per_window where K is no multiple of a cache line, so that contiguous rows
// start off the lines.  The plan knows no bases or pitches (the workspace has a size for M, N and K
// alone), so rows off the lines for another reason are counted as if on them; shifted() goes by them.
struct TileCost {
  int bm, bn;
  float fixed, per_window, again, off_lines;
};
// TILE_128x128_SHORT: rings of two windows, so that two workgroups fit a CU and one loads while the other
// stores (13986 x 416 x 1664: 31 -> 24 us); with a longer K the deeper ring is faster (1024 x 4096 x 4096:
// 31 us, 22.5).
constexpr int kShortWindows = 4;
constexpr float kLaunch = 3.0f, kDispatch = 1.07f;
enum { TILE_256x256, TILE_128x256, TILE_128x128, TILE_64x128, TILE_128x64, TILE_64x64, TILE_64x32, TILE_32x64, TILE_32x32, TILE_128x128_SHORT, TILES };
constexpr TileCost kTileCost[TILES] = {
    {256, 256, 12.2f, 1.156f, 1.0f, 1.3f},  {128, 256, 11.7f, 0.728f, 1.0f, 1.25f}, {128, 128, 6.5f, 0.537f, 1.0f, 1.06f},
    {64, 128, 5.8f, 0.404f, 1.0f, 1.06f},   {128, 64, 5.8f, 0.404f, 1.0f, 1.06f},   {64, 64, 4.2f, 0.288f, 0.75f, 1.06f},
    {64, 32, 4.0f, 0.222f, 0.75f, 1.06f},   {32, 64, 4.0f, 0.225f, 0.75f, 1.06f},   {32, 32, 3.2f, 0.162f, 0.75f, 1.06f},
    {128, 128, 6.05f, 0.59f, 0.75f, 1.06f}};
struct Plan {
  int tile, splits, tail;   // tail: the tile that the last round of 256 x 256 tiles is cut into, or -1
};
inline Plan plan_w8a8(int64_t M, int64_t N, int64_t K, bool may_split) {
  const int64_t nwin = (K + kWin - 1) / kWin;
  Plan best{TILE_256x256, 1, -1};
  double least = 0;
  auto consider = [&](double us, Plan plan) {
    if (least == 0 || us < least) {
      least = us;
      best = plan;
    }
  };
  auto round = [&](int t, int64_t windows) {
    const TileCost& c = kTileCost[t];
    return c.fixed - kLaunch + (K % kWin ? c.off_lines : 1.0f) * c.per_window * (double)windows;
  };
  for (int t = 0; t < TILES; ++t) {
    const TileCost& c = kTileCost[t];
    const int64_t tiles = ((M + c.bm - 1) / c.bm) * ((N + c.bn - 1) / c.bn);
    if (t != TILE_256x256 && tiles > ((int64_t)1 << 22)) continue;   // threads of a launch stay below 2^32
    if (t == TILE_128x128_SHORT && nwin > kShortWindows) continue;
    for (int s = 1; s <= (may_split ? kMaxSplits : 1); ++s) {
      if (s > 1 && (tiles * s > 256 || nwin < 8 * s)) break;
      const double further = (double)((tiles * s + 255) / 256 - 1);
      const double first = round(t, (nwin + s - 1) / s);
      double us = kLaunch + first + (c.again * first > kDispatch ? c.again * first : kDispatch) * further;
      if (s > 1) us += 4.5 + (double)s * (double)M * (double)N * 8.0 / 5e6;
      consider(us, {t, s, -1});
    }
    const int64_t rest = tiles % 256;
    if (t == TILE_256x256 && tiles > 256 && rest > 0 && rest <= 128)
      for (int tail = TILE_128x256; tail <= TILE_128x128; ++tail)
        if (rest * (tail == TILE_128x256 ? 2 : 4) <= 256)
          consider(kLaunch + round(t, nwin) * (double)(tiles / 256) + round(tail, nwin), {t, 1, tail});
  }
  return best;
}

// Whether the launch takes the shifted forms of the tiles (rows that do not all start on a cache
// line).  For K up to 1024 the plain tiles are as fast off the lines (700 x 400 x 2000: 6.3 us, shifted
// 6.5; 1001 x 1360 x 2051: 12.0 and 11.4, 1024 x 4112 x 4096: 32 and 23.5).
inline bool shifted(int64_t K, uintptr_t a, int64_t ld_a, uintptr_t w, int64_t ld_w) {
  return (K + kWin - 1) / kWin > 8 && ((a | (uintptr_t)ld_a | w | (uintptr_t)ld_w) % 128) != 0;
}

}  // namespace mxq
