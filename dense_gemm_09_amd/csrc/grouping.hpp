// Row groups of the grouped products: which tile of which group a workgroup computes.
#pragma once

#include "common.hpp"
#include "grouped_plan.hpp"

namespace g355 {

// Word 3 of a raw buffer descriptor on gfx9-family parts (32-bit data format,
// no swizzle, no index stride).
constexpr int kBufferWord3 = 0x00020000;

// ------------------------------------------------------- products grouped by rows

// MODE_GROUPED: rows offsets[g] .. offsets[g+1]-1 of A and C belong to group
// g, which has a B (bias, scale_b, sum_b) of its own. MODE_WGRAD: C of group g
// is the product of two operands over those rows (their contraction axis).
enum TileMode : int { MODE_DENSE = 0, MODE_GROUPED = 1, MODE_WGRAD = 2 };

// Tile rows that a group's tiles are numbered along before the next column: the
// tiles in flight on an XCD share that many row panels, and a group of that many
// tile rows has its weight read once (16384 x 14336 x 4096 over 8 experts, in one
// run: 1736 us with 2, 1645 with 4, 1617 with 8).
constexpr int kGroupedBand = 8;

// Group g's rows [s, e). The offsets are device data that no host check has
// seen: clamped here, so that whatever they hold no access leaves the arrays.
__device__ __forceinline__ void group_rows(const GemmArgs& p, int g, int& s, int& e) {
  s = min(max(p.offsets[g], 0), p.rows_total);
  e = min(max(p.offsets[g + 1], s), p.rows_total);
}

// The row tile of workgroup `b`: every wave counts the row tiles of all groups
// (64 groups at a time, one per lane) and finds its own in their running sum,
// so the launch needs neither a host copy of the offsets nor a kernel before
// it. The grid is the largest count possible; workgroups past the real one
// (nwg) return, and the real ones are spread over the XCDs evenly.
// tiles: row tiles of the found group; first: row tiles of the groups before it.
template <int BM>
__device__ __forceinline__ bool find_group(const GemmArgs& p, int b, int lane, int& L, int& g,
                                           int& s, int& rows, int& tiles, int& first) {
  const auto count = [&](int c, int& gs, int& ge) {
    gs = ge = 0;
    if (c + lane < p.groups) group_rows(p, c + lane, gs, ge);
    return (ge - gs + BM - 1) / BM;
  };
  const auto running_sum = [&](int n) {
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
      const int t = __shfl_up(n, o);
      n += lane >= o ? t : 0;
    }
    return n;
  };
  // The first 64 groups stay in registers for the second pass.
  int gs, ge;
  int n = count(0, gs, ge);
  int incl = running_sum(n);
  int64_t all = __builtin_amdgcn_readlane(incl, 63);
  for (int c = 64; c < p.groups; c += 64) {
    int cs, ce;
    all += __builtin_amdgcn_readlane(running_sum(count(c, cs, ce)), 63);
  }
  // Offsets that decrease can count more tiles than the grid has: nothing is
  // computed then (their result is undefined, and the sums below stay in range).
  if (all * p.tiles_n > static_cast<int64_t>(gridDim.x)) return false;
  const int nwg = static_cast<int>(all) * p.tiles_n;
  if (b >= nwg) return false;
  L = xcd_remap(b, nwg);
  const int rt = L / p.tiles_n;
  int before = 0;
  for (int c = 0; c < p.groups; c += 64) {
    if (c > 0) {
      n = count(c, gs, ge);
      incl = running_sum(n);
    }
    const unsigned long long hit = __ballot(before + incl > rt);
    if (hit != 0) {
      const int src = __builtin_ctzll(hit);
      g = c + src;
      s = __builtin_amdgcn_readlane(gs, src);
      rows = __builtin_amdgcn_readlane(ge, src) - s;
      tiles = __builtin_amdgcn_readlane(n, src);
      first = before + __builtin_amdgcn_readlane(incl, src) - tiles;
      return true;
    }
    before += __builtin_amdgcn_readlane(incl, 63);
  }
  return false;  // not reached: rt < all
}

// The groups' row tiles as a table in LDS, for workgroups that take many tiles.
struct GroupTable {
  int begin[kTableGroups], end[kTableGroups];  // rows
  int tiles[kTableGroups];                     // row tiles up to and with this group
  int row_tiles;                               // in all; 0 where the offsets count more than the launch has
};

// Filled by wave 0 (the caller's barrier follows).
template <int BM>
__device__ __forceinline__ void fill_table(const GemmArgs& p, GroupTable& t, int wave, int lane) {
  if (wave != 0) return;
  int before = 0;
  bool fits = true;
  for (int c = 0; c < p.groups; c += 64) {
    int s = 0, e = 0;
    if (c + lane < p.groups) group_rows(p, c + lane, s, e);
    int n = (e - s + BM - 1) / BM;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
      const int x = __shfl_up(n, o);
      n += lane >= o ? x : 0;
    }
    t.begin[c + lane] = s;
    t.end[c + lane] = e;
    t.tiles[c + lane] = before + n;
    before += __builtin_amdgcn_readlane(n, 63);
    // Offsets that decrease can count more tiles than the groups can have.
    fits = fits && static_cast<int64_t>(before) * p.tiles_n <= p.turn_tiles;
    if (!fits) break;
  }
  if (lane == 0) t.row_tiles = fits ? before : 0;
}

// The group of row tile `rt` < row_tiles, as in find_group.
__device__ __forceinline__ void find_in_table(const GroupTable& t, int rt, int groups, int lane, int& g, int& s,
                                              int& rows, int& tiles, int& first) {
  int c = 0, end = 0;
  unsigned long long hit = 0;
  for (; c < groups; c += 64) {
    end = t.tiles[c + lane];
    hit = __ballot(end > rt);
    if (hit != 0) break;
  }
  g = c + __builtin_ctzll(hit);
  first = __builtin_amdgcn_readfirstlane(g > 0 ? t.tiles[g - 1] : 0);
  tiles = __builtin_amdgcn_readfirstlane(t.tiles[g]) - first;
  s = __builtin_amdgcn_readfirstlane(t.begin[g]);
  rows = __builtin_amdgcn_readfirstlane(t.end[g]) - s;
}

// The tile of workgroup `b` of a weight gradient: every group has the same
// tiles, and the groups differ in their K range. Each XCD takes an eighth of
// every group's tiles, neighbours of each other, so that groups of unequal
// length load the XCDs alike.
__device__ __forceinline__ bool wgrad_tile(const GemmArgs& p, int b, int& g, int& tm, int& tn) {
  const int tiles = p.tiles_m * p.tiles_n;
  g = b / tiles;
  int t = b - g * tiles;
  if (tiles >= kWgradXcdTiles) {
    const int per = (tiles + 7) / 8;
    g = (b >> 3) / per;
    t = (b & 7) * per + (b >> 3) - g * per;
    if (t >= tiles) return false;
  }
  tile_coords(t, p.tiles_m, p.tiles_n, 4, tm, tn);
  return true;
}

}  // namespace g355
