// Block-128 FP8 products: out[r, n] = sum over K blocks kb of
//   sa[r, kb] sb[n / 128, kb] sum over k in kb of a[r, k] b[n, k]
// with E4M3 codes, FP32 scales, FP32 accumulation and one rounding of the
// result (dense, batch, grouped-contiguous, grouped-masked, and the
// form that sums over each group's range of K).
//
// A K block is one step: the matrix instruction sums the 128 products of a
// step from zero, and the vector unit adds that sum times sa sb to the FP32
// accumulator.  The scales are per row of a and per 128 columns, so a lane's
// factor is one product for all accumulators of its row.
#include "block_launch.hpp"
#include "hq.h"

namespace hq {
namespace {

// ------------------------------------------------------------------ direct
// Few rows: the weights are read once and bound the call.  A workgroup of W
// waves takes 16 MF rows x 16 NF columns of one batch item; its waves take runs
// of U K blocks in turn, each lane loading its operands from global memory (U
// blocks in flight), and their sums meet in LDS in wave order.  No LDS staging:
// a row's 128 codes are read once, in the lanes that multiply them.  Every wave
// that fits keeps loads under way: W = 16, U = 2 was the best of W 4 .. 16, U 1 ..
// 4.  1x17408x5120 takes 17.4 us where a part of the 89 MB of weights is still in
// the Infinity Cache (three sets of operands in turn), 20.2 us, 4.4 TB/s, where
// none is.  With more rows every workgroup's reads of A from the L2s and the
// widening of both operands show: 16 rows 27 and 30.5 us.  Narrow outputs leave
// units without work (1x1536x7168 6.6 us, 1.7 TB/s).  Non-temporal weight loads
// cost 1 to 17 %.
template <int MF, int NF, int W, int U>
__global__ __launch_bounds__(W * 64) void block_gemm_direct(BlockGemmArgs p) {
  __shared__ v4f part[W - 1][MF * NF][64];
  const int tid = threadIdx.x, lane = tid & 63, w = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int r16 = lane & 15, q = lane >> 4;
  const int64_t g = blockIdx.y, row0 = g * p.slot_rows, row_end = row0 + p.slot_rows;
  const int64_t n0 = (int64_t)blockIdx.x * 16 * NF;
  const float* sb = p.sb + (g * p.nnb + n0 / 128) * p.nkb;
  const uint8_t* bp[NF];
#pragma unroll
  for (int j = 0; j < NF; ++j) {
    const int64_t nb = n0 + 16 * j + r16;
    bp[j] = p.b + (g * p.n + (nb < p.n ? nb : p.n - 1)) * p.k + 16 * q;
  }
  const uint8_t* ap[MF];
  const float* sap[MF];
  v4f acc[MF][NF];
#pragma unroll
  for (int i = 0; i < MF; ++i) {
    const int64_t r = row0 + 16 * i + r16, rr = r < row_end ? r : row_end - 1;
    ap[i] = p.a + rr * p.k + 16 * q;
    sap[i] = p.sa + rr * p.nkb;
#pragma unroll
    for (int j = 0; j < NF; ++j) acc[i][j] = v4f{0, 0, 0, 0};
  }
  const int k16 = (int)p.k - 16 * q;           // codes of a row from the lane's first one on
  for (int kb = w * U; kb < p.nkb; kb += W * U) {
    v8i bf[NF][U], af[MF][U];
    float sv[U], sav[MF][U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int k0 = (kb + u) * 128;
#pragma unroll
      for (int j = 0; j < NF; ++j) bf[j][u] = load_pair(bp[j] + k0, k0 < k16, k0 + 64 < k16);
      sv[u] = kb + u < p.nkb ? sb[kb + u] : 0.0f;
#pragma unroll
      for (int i = 0; i < MF; ++i) {
        af[i][u] = load_pair(ap[i] + k0, k0 < k16, k0 + 64 < k16);
        sav[i][u] = kb + u < p.nkb ? sap[i][kb + u] : 0.0f;
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int i = 0; i < MF; ++i) {
        const float f = sav[i][u] * sv[u];
#pragma unroll
        for (int j = 0; j < NF; ++j) {
          const v4f t = dot16(bf[j][u], af[i][u]);
#pragma unroll
          for (int e = 0; e < 4; ++e) acc[i][j][e] = __builtin_fmaf(t[e], f, acc[i][j][e]);
        }
      }
  }
  if (w > 0) {
#pragma unroll
    for (int i = 0; i < MF * NF; ++i) part[w - 1][i][lane] = acc[i / NF][i % NF];
  }
  __syncthreads();
  if (w == 0) {
#pragma unroll
    for (int i = 0; i < MF * NF; ++i) {
      v4f v = acc[i / NF][i % NF];
#pragma unroll
      for (int o = 0; o < W - 1; ++o) v += part[o][i][lane];
      const int64_t r = row0 + 16 * (i / NF) + r16, n = n0 + 16 * (i % NF) + 4 * q;
      if (r < row_end && n < p.n) store4(p.out, p.out_kind, r * p.n + n, v);
    }
  }
}

// ------------------------------------------------------------------ K split
// out = the slices' FP32 partial sums [slices, rows, n], added in slice order:
// the same bits from run to run.  Its launch and the partials' way through the
// caches bound it.  Small sums load a thread's slices together: one at a time a
// call took 22.1 us instead of 21.5 (17x5120x17408), 12.3 instead of 11.3 (50x
// 1536x4096); loads past the last slice repeat it.  From 2^18 quads on other
// waves cover the loads, and together they cost 0.5 to 0.9 %.
constexpr int kReduceThreads = 256;
template <int FLIGHT>      // slices loaded at once
__global__ __launch_bounds__(kReduceThreads) void block_reduce(const float* __restrict__ partial, int slices,
                                                               int64_t rows, uint32_t nq, int64_t ldo, void* out,
                                                               int32_t kind) {
  const int64_t i = (int64_t)blockIdx.x * kReduceThreads + threadIdx.x, quads = rows * nq;
  if (i >= quads) return;
  const v4f* src = reinterpret_cast<const v4f*>(partial) + i;
  v4f v = {0, 0, 0, 0};
  for (int s0 = 0; s0 < slices; s0 += FLIGHT) {
    v4f x[FLIGHT];
#pragma unroll
    for (int s = 0; s < FLIGHT; ++s) x[s] = src[(s0 + s < slices ? s0 + s : slices - 1) * quads];
#pragma unroll
    for (int s = 0; s < FLIGHT; ++s)
      if (s0 + s < slices) v = s0 + s == 0 ? x[0] : v + x[s];
  }
  const int64_t row = i / nq;
  store4(out, kind, row * ldo + 4 * (i - row * nq), v);
}

hipError_t launch_tiled(hipStream_t s, BlockGemmArgs p, const DeviceInfo& dev, bool fast, const Plan& pl, void* ws) {
  const BlockGemmArgs whole = p;
  if (pl.slices > 1) {
    p.slices = pl.slices;
    p.out = ws;
    p.out_kind = kOutF32;
    p.ldo = p.n;
  }
  const int policy = plan_policy(p);
  const hipError_t e = fast ? launch_block_fast(s, p, dev, pl.tile, policy) : launch_block_exact(s, p, dev, pl.tile, policy);
  if (e != hipSuccess || pl.slices == 1) return e;
  const int64_t quads = p.rows * p.n / 4;
  const auto reduce = quads >= 1 << 18 || pl.slices == 2 ? block_reduce<2>
                      : pl.slices <= 4                   ? block_reduce<4>
                                                         : block_reduce<8>;
  hipLaunchKernelGGL(reduce, dim3((unsigned)up(quads, kReduceThreads)), dim3(kReduceThreads), 0, s,
                     static_cast<const float*>(ws), pl.slices, p.rows, (uint32_t)(p.n / 4), whole.ldo, whole.out,
                     whole.out_kind);
  return hipGetLastError();
}

}  // namespace

uint64_t block_gemm_workspace_bytes(const BlockGemmArgs& p, const DeviceInfo& dev) {
  return direct_path(p) ? 0 : plan_all(p, dev, fast_path(p), HQ_BLOCK_WORKSPACE_BYTES).bytes(p);
}

hipError_t launch_block_gemm(hipStream_t s, const BlockGemmArgs& args, const DeviceInfo& dev, void* workspace,
                             uint64_t workspace_bytes) {
  BlockGemmArgs p = args;
  p.ldo = p.n;
  if (direct_path(p)) {
    // 16-column workgroups, or 32-column ones where they are many: those read
    // A half as often (from 6 rows on: 16x17408x5120 30.3 -> 26.4 us, 1 row
    // 17.6 -> 19.3 us), and where 16 columns would make between one and two
    // workgroups per compute unit they share the work evenly
    // (1x5120x17408 22.9 -> 21.0 us, 16 rows 40.4 -> 30.5 us)
    const int64_t narrow = up(p.n, 16) * p.groups;
    if (narrow > dev.num_cus && (narrow < 2 * dev.num_cus || p.slot_rows >= 6))
      hipLaunchKernelGGL((block_gemm_direct<1, 2, 8, 2>), dim3((unsigned)up(p.n, 32), (unsigned)p.groups), dim3(512), 0,
                         s, p);
    else
      hipLaunchKernelGGL((block_gemm_direct<1, 1, 16, 2>), dim3((unsigned)up(p.n, 16), (unsigned)p.groups), dim3(1024), 0,
                         s, p);
    return hipGetLastError();
  }
  const bool fast = fast_path(p);
  if (p.form != kUniform) {
    Plan pl;
    pl.tile = plan_grouped(p, fast);
    return launch_tiled(s, p, dev, fast, pl, nullptr);
  }
  // the plan that HQ_BLOCK_WORKSPACE_BYTES would allow if the workspace holds
  // it, else the best one without a split
  Plans pl = plan_all(p, dev, fast, HQ_BLOCK_WORKSPACE_BYTES);
  if (pl.bytes(p) > (workspace != nullptr ? workspace_bytes : 0)) pl = plan_all(p, dev, fast, 0);
  if (pl.head == 0) return launch_tiled(s, p, dev, fast, pl.all, workspace);
  const int64_t head = pl.head;
  BlockGemmArgs first = p, rest = p;
  first.n = head;
  const hipError_t e = launch_tiled(s, first, dev, fast, pl.all, nullptr);
  if (e != hipSuccess) return e;
  rest.n = p.n - head;
  rest.b += head * p.k;
  rest.sb += head / 128 * p.nkb;
  rest.out = static_cast<uint8_t*>(p.out) + head * (p.out_kind == kOutF32 || p.out_kind == kOutF32Add ? 4 : 2);
  return launch_tiled(s, rest, dev, fast, pl.rest, workspace);
}

}  // namespace hq
