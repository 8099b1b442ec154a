// 16-bit products by expert: out[r] = a[r] b[g]^T (or a[r] b[g]) for the rows r
// of group g, and out[g] = sum over its rows of a[r]^T b[r].  The direct kernel
// for calls of few rows, and the choice of kernel and tile.
#include "group_tiles.hpp"
#include "half_launch.hpp"
#include "half_math.hpp"

namespace hq {
namespace {

// The group and rows of m-tile `mt` (16 rows); g < 0: there is no such tile.
__device__ __forceinline__ GroupTile direct_tile(const HalfGemmArgs& p, int mt) {
  if (p.form == kContiguous) return group_tile(p.group_end, p.groups, (int)p.rows, 16, mt);
  const int per = (int)((p.slot_rows + 15) / 16), g = mt / per;
  const int64_t v = p.counts[g], c = v < 0 ? 0 : (v > p.slot_rows ? p.slot_rows : v);
  GroupTile t{};
  t.row0 = (int)(g * p.slot_rows) + (mt - g * per) * 16;
  t.row_end = (int)(g * p.slot_rows + c);
  t.g = t.row0 < t.row_end ? g : -1;
  return t;
}

// A workgroup of W waves takes 16 rows x 16 columns; its waves take runs of U x 64
// K values in turn, each lane loading its operands from memory, and their sums
// meet in LDS in the order of the waves.  The weights' stream bounds it: 8 rows
// of 8 experts of 1536 x 2048 13.1 us (50 MB, 3.8 TB/s, the launch and the search
// for the group among them), 4 tokens and 8 of 64 experts of 2048 x 4096 63 us.
// Against it: 16 waves 14.9 and 72 us; 4 runs in flight 13.0 and 64 us; 32 columns a
// workgroup 12.7 and 73 us; 4 waves of 4 runs 13.5 and 66 us.
template <bool F16, int W, int U>
__global__ __launch_bounds__(W * 64) void half_gemm_direct(HalfGemmArgs p) {
  __shared__ v4f part[W - 1][64];
  const GroupTile t = direct_tile(p, blockIdx.y);
  if (t.g < 0) return;
  const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int x = lane & 15, q = lane >> 4, k = (int)p.k;
  const int64_t n0 = (int64_t)blockIdx.x * 16, nb = n0 + x < p.n ? n0 + x : p.n - 1;
  const bool live = t.row0 + x < t.row_end;
  const uint16_t* bp = p.b + ((int64_t)t.g * p.n + nb) * p.k + 8 * q;
  const uint16_t* ap = p.a + (int64_t)(live ? t.row0 + x : t.row0) * p.k + 8 * q;
  v4f acc = {0, 0, 0, 0};
  const int kq = k - 8 * q;                // values of a row from the lane's first one on
  for (int k0 = w * U * 64; k0 < k; k0 += W * U * 64) {
    v4i bf[U][2], af[U][2];
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int at = k0 + u * 64 + h * 32;
        bf[u][h] = af[u][h] = v4i{0, 0, 0, 0};
        if (at < kq) bf[u][h] = *reinterpret_cast<const v4i*>(bp + at);
        if (at < kq && live) af[u][h] = *reinterpret_cast<const v4i*>(ap + at);
      }
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int h = 0; h < 2; ++h) acc = product16<F16>(bf[u][h], af[u][h], acc);
  }
  if (w > 0) part[w - 1][lane] = acc;
  __syncthreads();
  if (w > 0) return;
#pragma unroll
  for (int i = 0; i < W - 1; ++i) acc += part[i][lane];
  if (live && n0 + 4 * q < p.n) store4(p.out, p.out_kind, (int64_t)(t.row0 + x) * p.n + n0 + 4 * q, acc);
}

constexpr int kDirectWaves = 8, kDirectUnroll = 2;
hipError_t launch_direct(hipStream_t s, const HalfGemmArgs& p, int64_t mt) {
  const dim3 grid((unsigned)((p.n + 15) / 16), (unsigned)mt), block(kDirectWaves * 64);
  if (p.f16) hipLaunchKernelGGL((half_gemm_direct<true, kDirectWaves, kDirectUnroll>), grid, block, 0, s, p);
  else hipLaunchKernelGGL((half_gemm_direct<false, kDirectWaves, kDirectUnroll>), grid, block, 0, s, p);
  return hipGetLastError();
}

// At most this many 16-row m-tiles.
int64_t direct_tiles(const HalfGemmArgs& p) {
  return p.form == kMasked ? (p.slot_rows + 15) / 16 * p.groups : p.rows / 16 + (p.rows < p.groups ? p.rows : p.groups);
}

constexpr int kDirect = -1;      // not a tile: the direct kernel

// Results that the L2s cannot hold leave past them, and the operands stay: 65536
// rows x 4096 688 -> 685 us, their sums for the weights (805 MB) 737 -> 722 us, 402 MB
// of such sums 215 -> 219 us, 100 MB as 16 bits (3440 x 1088) 90 -> 82 us.  Only where
// every row starts a line: lines written in two parts need the L2s (377 MB of 1072 x
// 2312 FP32 sums 111 -> 152 us past them).
bool plan_stream(const HalfGemmArgs& p) {
  const int64_t wide = p.out_kind >= kOutF32 ? 4 : 2, bytes = (p.form == kGroupK ? p.groups : 1) * p.rows * p.n * wide;
  return bytes > (int64_t)32 << 20 && p.n * wide % 128 == 0 && (uintptr_t)p.out % 128 == 0;
}

// The kernel and tile of a call, by the rows a group has on average (only the
// device knows them).  Measured in us, 64 experts of 2048 x 4096 in BF16, T tokens
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
int plan_half(const HalfGemmArgs& p, const DeviceInfo& dev) {
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

}  // namespace

hipError_t launch_half_gemm(hipStream_t s, const HalfGemmArgs& args, const DeviceInfo& dev) {
  HalfGemmArgs p = args;
  p.stream = plan_stream(p);
  const int tile = plan_half(p, dev);
  if (p.form == kGroupK) return launch_half_tn(s, p, dev, tile);
  if (tile == kDirect) return launch_direct(s, p, direct_tiles(p));
  return p.b_t ? launch_half_nn(s, p, dev, tile) : launch_half_nt(s, p, dev, tile);
}

}  // namespace hq
