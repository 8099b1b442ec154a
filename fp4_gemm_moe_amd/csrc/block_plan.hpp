// Which kernel, tile shape and K split a block-128 FP8 product takes: rules on
// its form, sizes and result type, host code only.
#pragma once

#include <algorithm>

#include "block_internal.hpp"

namespace hq {

// BF16 results of four K blocks or more take the FP8 matrix instructions: their
// sums are off by 1.5e-5 of the norm at K = 128 and less with every further
// block, a hundredth of the BF16 rounding at four.  Shorter sums, and FP16 and
// FP32 results, go through FP16 operands with full FP32 sums.  So do sums over
// the groups' ranges of K: only the device knows their lengths, and one of a
// single block has no further ones to average over.
inline bool fast_path(const BlockGemmArgs& p) { return p.out_kind == kOutBf16 && p.nkb >= 4 && p.form != kGroupK; }

// Tile shapes of the tiled kernel (rows x columns).
enum BlockTile : int { kTile256x256, kTile256x128, kTile128x256, kTile128x128, kTile64x128 };

// A tile shape and what one of its steps takes (microseconds), fitted to calls
// of 17 to 4096 rows over 17408 x 5120 and 5120 x 17408.  A step costs less
// where tiles share their weights on a full chip (256x256 2.10, 128x256 1.12,
// 128x128 0.71, 64x128 0.48 at 4096 x 4096 x 4096) and where part of the chip
// idles (256x256 1.47 at half of it); a model with both chose worse over 38
// shapes (2048x17408x5120 189 -> 233 us, 128x17408x5120 36 -> 52 us).
struct Shape {
  int tile, bm, bn;
  double us;
};
constexpr Shape kFast[] = {{kTile256x256, 256, 256, 2.13}, {kTile128x256, 128, 256, 1.30},
                           {kTile128x128, 128, 128, 0.80}, {kTile64x128, 64, 128, 0.65}};
constexpr Shape kExact[] = {{kTile256x128, 256, 128, 1.95}, {kTile128x128, 128, 128, 1.40}, {kTile64x128, 64, 128, 0.90}};

constexpr double kBytesPerUs = 5.0e6;      // HBM, of the partial sums and of weights that are read once
constexpr double kLaunchUs = 3.0;          // a further launch on the stream

// How a launch over n columns is tiled, and its estimated time.
struct Plan {
  int tile = kTile256x256;
  int slices = 1;
  double us = 1e30;
  uint64_t bytes(int64_t rows, int64_t n) const { return slices > 1 ? (uint64_t)slices * rows * n * 4 : 0; }
};

inline int64_t up(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Uniform rows: the shape and K split with the least estimated time, rounds of
// the chip x steps x step time, plus what writing, reading and adding up the
// partial sums takes.  A step whose weights no other m-tile shares takes at
// least their time from memory.
inline Plan plan_uniform(const BlockGemmArgs& p, int64_t n, const DeviceInfo& dev, bool fast, uint64_t ws) {
  Plan best;
  const int64_t cus = dev.num_cus;
  auto consider = [&](const Shape& sh) {
    const int64_t mt = up(p.slot_rows, sh.bm), tiles = mt * p.groups * up(n, sh.bn);
    for (int s = 1; s <= 16 && (s == 1 || s * 4 <= p.nkb); ++s) {
      Plan c;
      c.tile = sh.tile;
      c.slices = s;
      if (c.bytes(p.rows, n) > ws) break;
      const double stream = mt == 1 ? sh.bn * 128.0 * std::min(tiles * s, cus) / kBytesPerUs : 0.0;
      c.us = up(up(tiles * s, 8), cus / 8) * up(p.nkb, s) * std::max(sh.us, stream);
      if (s > 1) c.us += kLaunchUs + 2.0 * c.bytes(p.rows, n) / kBytesPerUs;
      if (c.us < best.us) best = c;
    }
  };
  if (fast) for (const Shape& sh : kFast) consider(sh);
  else for (const Shape& sh : kExact) consider(sh);
  return best;
}

// One launch over all columns, or two: whole rounds of 256 x 256 tiles over
// the first `head` columns, then the rest in smaller tiles or K slices, where
// that is done sooner than a partly filled last round.
struct Plans {
  Plan all, rest;
  int64_t head = 0;      // 0: one launch
  uint64_t bytes(const BlockGemmArgs& p) const { return head > 0 ? rest.bytes(p.rows, p.n - head) : all.bytes(p.rows, p.n); }
};

inline Plans plan_all(const BlockGemmArgs& p, const DeviceInfo& dev, bool fast, uint64_t ws) {
  Plans pl;
  pl.all = plan_uniform(p, p.n, dev, fast, ws);
  if (!fast || p.groups != 1 || pl.all.tile != kTile256x256 || pl.all.slices != 1) return pl;
  const int64_t mt = up(p.slot_rows, 256), nt = up(p.n, 256), cus = dev.num_cus;
  const int64_t rounds = mt * nt / cus, head = rounds * cus / mt;
  if (rounds < 1 || head < 1 || head >= nt) return pl;
  pl.rest = plan_uniform(p, p.n - head * 256, dev, fast, ws);
  const double us = up(up(mt * head, 8), cus / 8) * p.nkb * kFast[0].us + kLaunchUs + pl.rest.us;
  if (us < 0.97 * pl.all.us) pl.head = head * 256;
  return pl;
}

// Grouped forms, by the rows a group has (on average where only the device
// knows them): few rows leave the weights' stream to bound the call, which the
// deeper stages of the smaller tiles serve better; many share each weight tile.
// Measured in us, K = 2048 and 4096, N = 4096: 32 slots of 64 rows 111 (64x128),
// 122 (128x256), of 128 rows 169, 126, of 256 rows 174 (128x256), 138 (256x256);
// contiguous groups of 256 rows on average 66.5 (128x256), 69 (256x256), of 512
// rows 101, 95, of 1024 rows 175, 160.
inline int plan_grouped(const BlockGemmArgs& p, bool fast) {
  const int64_t per = p.form == kContiguous ? up(p.rows, p.groups) : (p.form == kGroupK ? p.rows : p.slot_rows);
  if (per <= (p.form == kMasked ? 64 : 32)) return kTile64x128;
  if (!fast) return per <= 128 ? kTile128x128 : kTile256x128;
  return per <= (p.form == kContiguous ? 384 : 128) ? kTile128x256 : kTile256x256;
}

// The policy (BlockPolicy) of one tiled launch, p as it is launched.  Results
// that the L2s cannot hold leave past them, and the operands stay
// (4096x17408x5120 371 -> 357 us, FP32 K-grouped 971 -> 925 us); partial sums
// and smaller results are read again soon.  Masked slots of at most 256 rows
// read each weight once, by all compute units at once: those loads stream too
// (64 slots of 256 rows, 4096x7168: 513 -> 473 us).
inline int plan_policy(const BlockGemmArgs& p) {
  const int64_t bytes = (p.form == kGroupK ? p.groups : 1) * p.rows * p.n * (p.out_kind >= kOutF32 ? 4 : 2);
  if (p.form == kMasked && p.slot_rows <= 256) return kPolStreamAll;
  return p.slices == 1 && bytes > (int64_t)32 << 20 ? kPolStreamOut : kPolKeep;
}

// At most 16 rows, and columns that fit one launch (1024 threads for 16 of them).
inline bool direct_path(const BlockGemmArgs& p) {
  return p.form == kUniform && p.slot_rows <= 16 && up(p.n, 16) <= (kMaxWorkItems - 1) / 1024;
}

}  // namespace hq
