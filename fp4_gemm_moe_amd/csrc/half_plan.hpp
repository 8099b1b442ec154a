// Which kernel and tile shape a 16-bit product takes, and whether its results leave
// past the caches: rules on its form, sizes and result type, host code only.
#pragma once

#include "half_internal.hpp"

namespace hq {

// Tile shapes of the tiled kernel (rows x columns); kDirect: the direct kernel.
enum HalfTile : int { kDirect = -1, kHalf256x256, kHalf128x256, kHalf128x128, kHalf64x128, kHalf32x64 };

// At most this many 16-row m-tiles.
inline int64_t direct_tiles(const HalfGemmArgs& p) {
  return p.form == kMasked ? (p.slot_rows + 15) / 16 * p.groups : p.rows / 16 + (p.rows < p.groups ? p.rows : p.groups);
}

// Results that the L2s cannot hold leave past them, and the operands stay: 65536
// rows x 4096 688 -> 685 us, their sums for the weights (805 MB) 737 -> 722 us, 402 MB
// of such sums 215 -> 219 us, 100 MB as 16 bits (3440 x 1088) 90 -> 82 us.  Only where
// every row starts a line: lines written in two parts need the L2s (377 MB of 1072 x
// 2312 FP32 sums 111 -> 152 us past them).
inline bool plan_stream(const HalfGemmArgs& p) {
  const int64_t wide = p.out_kind >= kOutF32 ? 4 : 2, bytes = (p.form == kGroupK ? p.groups : 1) * p.rows * p.n * wide;
  return bytes > (int64_t)32 << 20 && p.n * wide % 128 == 0 && (uintptr_t)p.out % 128 == 0;
}

// The kernel and tile of a call, by the rows a group has on average (only the
// device knows them; where most groups are empty the tiles are too small: 1000 rows of
// 2048 x 4096 in two groups take 32.6 us as two groups and 65.4 as two of 64).  Measured in us, 64 experts of 2048 x 4096 in BF16, T tokens
// and 8 of the experts each; masked: 32 slots, 4096 x 2048.
//  - Few rows: the weights' stream bounds the call, and smaller tiles keep more
//    loads under way.  Direct / 32x64 / 64x128: T = 1 27.0 / 28.1 / 40.6, T = 16
//    108 / 121 / 139, slots of 8 99 / 104 / 108, of 16 111 / 102 / 110, of 32 -
//    / 103 / 112, of 64 - / 109 / 104; T = 64 - / 177 / 205.  With b [k, n]
//    (32x64 / 64x128) T = 1 32 / 44, T = 64 186 / 177: the small tile only where
//    the larger ones are few.
//  - More: rounds of the chip times what a tile takes.  A 128x128 tile takes 0.37 of a
//    256x256 one (0.28 to 0.47 over many shapes): T = 512 229 (128x128), 284
//    (256x256), T = 1024 300, 303, T = 2048 424, 398; 8 groups of 1900 rows, 648 x
//    3128, b [k, n]: 119, 89; slots of 128 rows 119, 138.  Sums over the groups' rows
//    0.32, since uneven groups leave more of the chip idle in tiles that are few: 10
//    groups, 18369 rows, 1288 x 584: 52, 88; 8 groups of 128 rows, 1024 x 768: 13.6,
//    17.4; 31 groups, 21162 rows, 5320 x 1288: 460, 340.
//  - Between them 128x256 tiles, for rows only, at 0.65 of a large one: 954 rows of 9
//    groups, 4192 x 816: 27.6 (256x256), 19.5, 23.0 (128x128); 1589 of 14, 5856 x 5328,
//    b [k, n]: 222, 280 (128x128).  Not where groups have up to 64 rows, each weight is
//    read once and two stages keep too few loads under way: T = 512 255, 229
//    (128x128); nor for sums (8056 rows of 12 groups, 2344 x 4432: 288, 236 (256x256)).
inline int plan_half(const HalfGemmArgs& p, const DeviceInfo& dev) {
  const int64_t cus = dev.num_cus;
  auto up = [](int64_t a, int64_t b) { return (a + b - 1) / b; };
  auto tiles = [&](int64_t bm, int64_t bn) -> int64_t {
    if (p.form == kGroupK) return up(p.rows, bm) * up(p.n, bn) * p.groups;
    if (p.form == kMasked) return up(up(p.slot_rows, 2) + bm / 2, bm) * p.groups * up(p.n, bn);
    return (p.rows / bm + up(p.rows < p.groups ? p.rows : p.groups, 2)) * up(p.n, bn);
  };
  if (p.form != kGroupK) {
    const bool masked = p.form == kMasked;
    const int64_t per = masked ? p.slot_rows : up(p.rows, p.groups);
    if (!p.b_t && per <= (masked ? 8 : 4) && direct_tiles(p) <= 65535) return kDirect;
    if (per <= (masked ? 32 : 16) && (!p.b_t || tiles(64, 128) <= 2 * cus)) return kHalf32x64;
    if (per <= (masked ? 64 : 32)) return kHalf64x128;
  }
  const double large = (double)up(tiles(256, 256), cus), small = (p.form == kGroupK ? 0.32 : 0.37) * up(tiles(128, 128), cus);
  if (p.form != kGroupK && (p.form == kMasked ? p.slot_rows / 2 : p.rows / p.groups) > 64) {
    const double half = 0.65 * up(tiles(128, 256), cus);
    if (half < large && half < small) return kHalf128x256;
  }
  return small < large ? kHalf128x128 : kHalf256x256;
}

}  // namespace hq
