// Tiles of rows of groups that lie one after another, found by every wave on its
// own: a lane has a run of at most 16 groups, and the wave's lanes scan them.
// Group ends are clamped as load_clamped_ends does it.
#pragma once

#include "sched.hpp"

namespace hq {

struct GroupTile {
  int g;                 // the group; -1: there is none
  int row0, row_end;     // the tile's first row, the group's end
  int index, first;      // the tile's number among all, and that of its group's first one
};

// Inclusive scans over a wave's lanes of non-negative values, by DPP moves: within
// rows of 16 lanes, then each row's last lane into the rows behind it.
template <class Op>
__device__ __forceinline__ int wave_scan(int v, Op op) {
  v = op(v, __builtin_amdgcn_update_dpp(0, v, 0x111, 0xf, 0xf, false));      // row_shr:1
  v = op(v, __builtin_amdgcn_update_dpp(0, v, 0x112, 0xf, 0xf, false));      // row_shr:2
  v = op(v, __builtin_amdgcn_update_dpp(0, v, 0x114, 0xf, 0xf, false));      // row_shr:4
  v = op(v, __builtin_amdgcn_update_dpp(0, v, 0x118, 0xf, 0xf, false));      // row_shr:8
  v = op(v, __builtin_amdgcn_update_dpp(0, v, 0x142, 0xa, 0xf, false));      // row_bcast:15, rows 1 and 3
  return op(v, __builtin_amdgcn_update_dpp(0, v, 0x143, 0xc, 0xf, false));   // row_bcast:31, rows 2 and 3
}
// The value of the lane before, 0 in the first.
__device__ __forceinline__ int lane_before(int v) { return __builtin_amdgcn_update_dpp(0, v, 0x138, 0xf, 0xf, false); }

// The last group's end.
__device__ __forceinline__ int last_end(const int32_t* __restrict__ ends, int groups, int rows) {
  int top = 0;
  for (int g = threadIdx.x & 63; g < groups; g += 64) top = ends[g] > top ? ends[g] : top;
  top = __builtin_amdgcn_readlane(wave_scan(top, OpMax()), 63);
  return top < rows ? top : rows;
}

// Tile number `want` of bm rows (by_group: the first tile of group `want`, with
// row0 its start, also where it is empty).  Uniform arguments; every lane of the
// wave gets the result.
template <bool by_group = false>
__device__ __forceinline__ GroupTile group_tile(const int32_t* __restrict__ ends, int groups, int rows, int bm, int want) {
  const int lane = threadIdx.x & 63, per = (groups + 63) / 64;
  int top = 0;
  for (int i = 0; i < per; ++i) {
    const int g = lane * per + i, e = g < groups ? ends[g] : 0;
    top = e > top ? e : top;
  }
  const int upto_end = wave_scan(top, OpMax()), before = lane_before(upto_end);
  // the run's groups: start and end of each from the largest end so far
  auto walk = [&](auto f) {
    int prev = before;
    for (int i = 0; i < per; ++i) {
      const int g = lane * per + i;
      if (g >= groups) break;
      const int e = ends[g], start = prev < rows ? prev : rows;
      prev = e > prev ? e : prev;
      const int end = prev < rows ? prev : rows;
      if (f(g, start, end, (end - start + bm - 1) / bm)) break;
    }
  };
  int tiles = 0;
  walk([&](int, int, int, int n) { tiles += n; return false; });
  const int upto = wave_scan(tiles, OpAdd());
  const int owner = by_group ? want / per : __popcll(__ballot(upto <= want));
  GroupTile t{-1, 0, 0, want, 0};
  if (owner >= 64) return t;
  int index = upto - tiles;
  if (lane == owner)
    walk([&](int g, int start, int end, int n) {
      if (by_group ? g == want : want < index + n) {
        t.g = g;
        t.row0 = by_group ? start : start + (want - index) * bm;
        t.row_end = end;
        t.first = index;
        return true;
      }
      index += n;
      return false;
    });
  t.g = __builtin_amdgcn_readlane(t.g, owner);
  t.row0 = __builtin_amdgcn_readlane(t.row0, owner);
  t.row_end = __builtin_amdgcn_readlane(t.row_end, owner);
  t.first = __builtin_amdgcn_readlane(t.first, owner);
  return t;
}

}  // namespace hq
