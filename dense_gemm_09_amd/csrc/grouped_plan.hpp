// Tiles and launch sizes of the products grouped by rows and of their weight
// gradient. Host arithmetic only, without HIP.
#pragma once

#include <algorithm>
#include <cstdint>

namespace g355 {

struct GroupedPlan {
  int bm, bn;    // tile
  int64_t grid;  // workgroups
};

// Groups that gemm_turn.hip's table of them holds (a multiple of 64).
constexpr int kTableGroups = 1024;

// Tiles per group from which the weight gradient deals each group's tiles to
// the XCDs in eighths (below, workgroups go round robin: an eighth of fewer
// tiles than this shares little).
constexpr int kWgradXcdTiles = 64;

constexpr int kGroupedCUs = 256;

inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Workgroups of a launch over row tiles of bm rows: the most that T rows in
// min(G, T) non-empty groups can need (each group may waste a partial tile).
inline int64_t most_row_tiles(int64_t G, int64_t T, int64_t bm) {
  return std::min(T, (T + std::min(G, T) * (bm - 1)) / bm);
}

// Tile of a grouped product. A group of `avg` rows takes avg / bm full tiles
// and on average half of one more. The costs are microseconds per 128-byte K
// slice of the slowest CU, from 180 shapes (2 to 32 groups of 32 to 400 rows,
// N = 1024 and 4096, K = 2048 and 7168, the three types): one tile's slice
// takes 0.65 us at 64x128 (ring of six slices), 0.72 at 128x128, 1.5 at 256x256; two
// 128x128 tiles on a CU 1.2, two 64x128 tiles 1.05. With B read along its rows, 0.9
// at 128x128 and 0.95 at 64x128 (two: 1.3): no kernel of 64 rows there, as 128 rows
// are never more workgroups. Examples, us at 64x128 / 128x128 / 256x256: BF16, 32
// groups of 400 rows, 4096 x 7168, 1715 / 1040 / 824; 8 groups of 200, 4096 x
// 2048, 94 / 40 / 53; 24 groups of a row or two, 2048 x 4096, 64.8 / 78.3; INT8,
// 30 groups of 4 rows, 4096 x 2048, 47 / 55, of 50 rows 63 / 60.
inline GroupedPlan plan_grouped(int64_t G, int64_t T, int64_t N, bool b_rows) {
  const double groups = static_cast<double>(std::min(G, T));
  const double avg = static_cast<double>(T) / groups;
  const auto workgroups = [&](int bm, int bn) {
    const double row_tiles = avg > 0.5 * bm ? avg / bm + 0.5 : 1.0;
    return groups * row_tiles * static_cast<double>(ceil_div(N, bn));
  };
  // Rounds of the CUs' slots; a last, partial round costs more than its share.
  const auto rounds = [](double wgs, double slots) {
    return wgs <= slots ? 1.0 : wgs / slots + 0.2;
  };
  const double w128 = workgroups(128, 128);
  const double w64 = workgroups(64, 128);
  const double c64 = b_rows              ? 1e30
                     : w64 <= kGroupedCUs ? 0.65
                                          : rounds(w64, 2 * kGroupedCUs) * 1.05;
  const double c128 = w128 <= kGroupedCUs ? (b_rows ? 0.9 : 0.72) : rounds(w128, 2 * kGroupedCUs) * 1.2;
  const double c256 = G <= kTableGroups ? rounds(workgroups(256, 256), kGroupedCUs) * 1.5 : 1e30;
  GroupedPlan best = c64 <= std::min(c128, c256) ? GroupedPlan{64, 128, 0}
                     : c128 <= c256              ? GroupedPlan{128, 128, 0}
                                                 : GroupedPlan{256, 256, 0};
  best.grid = most_row_tiles(G, T, best.bm) * ceil_div(N, best.bn);
  return best;
}

// Tile of the weight gradient: G equal grids of N x K outputs, in rounds of the
// CUs' slots. Measured, us at 256x256 / 128x128: 8 gradients of 14336 x 4096 over
// 16384 rows 1830 / 2149; 32 of 1000 x 2048 over 777 rows 40 / 53; 1 of 4096 x
// 4096 over 2000 rows 59 / 75; 4 of 1024 x 1024 over 4000 rows 38 / 22.
inline GroupedPlan plan_wgrad(int64_t G, int64_t N, int64_t K) {
  const auto cost = [&](int b, int occupancy, double eff) {
    const int64_t wgs = G * ceil_div(N, b) * ceil_div(K, b);
    return static_cast<double>(ceil_div(wgs, kGroupedCUs * occupancy)) * b * b * occupancy / eff;
  };
  const int b = cost(256, 1, 0.85) < cost(128, 2, 0.67) ? 256 : 128;
  const int64_t tiles = ceil_div(N, b) * ceil_div(K, b);
  return {b, b, G * (tiles >= kWgradXcdTiles ? 8 * ceil_div(tiles, 8) : tiles)};
}

}  // namespace g355
