// 16-bit products by expert: out[r] = a[r] b[g]^T (or a[r] b[g]) for the rows r
// of group g, and out[g] = sum over its rows of a[r]^T b[r].  The direct kernel
// for calls of few rows, and the choice of kernel and tile.
#include "half_launch.hpp"

namespace hq {
namespace {

typedef __bf16 v8b __attribute__((ext_vector_type(8)));

template <bool F16>
__device__ __forceinline__ v4f product16(v4i w, v4i x, v4f c) {
  if constexpr (F16)
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(v8h, w), __builtin_bit_cast(v8h, x), c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(v8b, w), __builtin_bit_cast(v8b, x), c, 0, 0, 0);
}

// The group and rows of m-tile `mt` (16 rows) of the groups, found by each wave
// on its own: a lane has a run of at most 16 groups.  g < 0: there is no such tile.
struct DirectTile {
  int g, row0, row_end;
};
__device__ __forceinline__ DirectTile direct_tile(const HalfGemmArgs& p, int mt) {
  const int lane = threadIdx.x & 63, per = (p.groups + 63) / 64;
  const bool masked = p.form == kMasked;
  int top = 0, tiles = 0;
  // the largest end of the lane's run, and of those before it (clamped ends never decrease)
  if (!masked) {
    for (int i = 0; i < per; ++i) {
      const int g = lane * per + i, e = g < p.groups ? p.group_end[g] : 0;
      top = e > top ? e : top;
    }
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) {
      const int v = __shfl_up(top, off, 64);
      if (lane >= off && v > top) top = v;
    }
    top = __shfl_up(top, 1, 64);
    if (lane == 0) top = 0;
  }
  const int rows = (int)p.rows;
  auto span = [&](int g, int& prev, int& start, int& end) {       // rows of group g; prev: the end before it
    if (masked) {
      const int64_t v = p.counts[g], c = v < 0 ? 0 : (v > p.slot_rows ? p.slot_rows : v);
      start = (int)(g * p.slot_rows);
      end = start + (int)c;
    } else {
      const int e = p.group_end[g];
      start = prev < rows ? prev : rows;
      prev = e > prev ? e : prev;
      end = prev < rows ? prev : rows;
    }
  };
  int prev = top, start, end;
  for (int i = 0; i < per; ++i) {
    const int g = lane * per + i;
    if (g >= p.groups) break;
    span(g, prev, start, end);
    tiles += (end - start + 15) / 16;
  }
  int upto = tiles;
#pragma unroll
  for (int off = 1; off < 64; off <<= 1) {
    const int v = __shfl_up(upto, off, 64);
    if (lane >= off) upto += v;
  }
  const int owner = __popcll(__ballot(upto <= mt));
  if (owner >= 64) return {-1, 0, 0};
  DirectTile t{-1, 0, 0};
  if (lane == owner) {
    int left = mt - (upto - tiles);
    prev = top;
    for (int i = 0; i < per; ++i) {
      const int g = lane * per + i;
      span(g, prev, start, end);
      const int n = (end - start + 15) / 16;
      if (left < n) {
        t = {g, start + left * 16, end};
        break;
      }
      left -= n;
    }
  }
  t.g = __builtin_amdgcn_readlane(t.g, owner);
  t.row0 = __builtin_amdgcn_readlane(t.row0, owner);
  t.row_end = __builtin_amdgcn_readlane(t.row_end, owner);
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
  const DirectTile t = direct_tile(p, blockIdx.y);
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

// The kernel and tile of a call, by the rows a group has on average (only the
// device knows them).  Measured in us, 64 experts of 2048 x 4096 in BF16, T tokens
// and 8 of the experts each; masked: 32 slots, 4096 x 2048.
//  - Few rows: the weights' stream bounds the call, and smaller tiles keep more
//    loads under way.  Direct / 32x64 / 64x128: T = 1 27.0 / 28.1 / 40.6, T = 16
//    108 / 121 / 139, slots of 8 99 / 104 / 108, of 16 111 / 102 / 110, of 32 -
//    / 103 / 112, of 64 - / 109 / 104; T = 64 - / 177 / 205.  With b [k, n]
//    (32x64 / 64x128) T = 1 32 / 44, T = 64 186 / 177: the small tile only where
//    the larger ones are few.
//  - More: rounds of the chip times what a tile takes.  A 128x128 tile takes 0.32 of a
//    256x256 one: T = 512 229 (128x128), 284 (256x256), T = 1024 300, 303, T = 2048
//    424, 398; slots of 128 rows 119, 138; sums over the groups' rows, 8 groups of
//    128 rows, 1024 x 768: 13.6, 17.4; 64 of 256 rows, 2048 x 1536: 317, 260.
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
  return 0.32 * up(tiles(128, 128), cus) < up(tiles(256, 256), cus) ? kHalf128x128 : kHalf256x256;
}

}  // namespace

hipError_t launch_half_gemm(hipStream_t s, const HalfGemmArgs& p, const DeviceInfo& dev) {
  const int tile = plan_half(p, dev);
  if (p.form == kGroupK) return launch_half_tn(s, p, dev, tile);
  if (tile == kDirect) return launch_direct(s, p, direct_tiles(p));
  return p.b_t ? launch_half_nn(s, p, dev, tile) : launch_half_nt(s, p, dev, tile);
}

}  // namespace hq
