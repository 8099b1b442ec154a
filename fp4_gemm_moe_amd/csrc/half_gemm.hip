// 16-bit products by expert: out[r] = a[r] b[g]^T (or a[r] b[g]) for the rows r
// of group g, and out[g] = sum over its rows of a[r]^T b[r].  The direct kernel
// for calls of few rows, and the launch that half_plan.hpp chooses.
#include "group_tiles.hpp"
#include "half_launch.hpp"
#include "half_math.hpp"
#include "half_plan.hpp"

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
