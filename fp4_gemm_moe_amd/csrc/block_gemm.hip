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
#include <algorithm>

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
// 4 (1x17408x5120 17.6 us, 5.1 TB/s of weights, a large copy's rate; 16 rows of
// A from the L2s take it to 26 us).  Non-temporal weight loads cost 1 to 17 %.
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

// ------------------------------------------------------------------ plan
// BF16 results of four K blocks or more take the FP8 matrix instructions: their
// sums are off by 1.5e-5 of the norm at K = 128 and less with every further
// block, a hundredth of the BF16 rounding at four.  Shorter sums, and FP16 and
// FP32 results, go through FP16 operands with full FP32 sums.  So do sums over
// the groups' ranges of K: only the device knows their lengths, and one of a
// single block has no further ones to average over.
bool fast_path(const BlockGemmArgs& p) { return p.out_kind == kOutBf16 && p.nkb >= 4 && p.form != kGroupK; }

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

int64_t up(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Uniform rows: the shape and K split with the least estimated time, rounds of
// the chip x steps x step time, plus what writing, reading and adding up the
// partial sums takes.  A step whose weights no other m-tile shares takes at
// least their time from memory.
Plan plan_uniform(const BlockGemmArgs& p, int64_t n, const DeviceInfo& dev, bool fast, uint64_t ws) {
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

Plans plan_all(const BlockGemmArgs& p, const DeviceInfo& dev, bool fast, uint64_t ws) {
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
int plan_grouped(const BlockGemmArgs& p, bool fast) {
  const int64_t per = p.form == kContiguous ? up(p.rows, p.groups) : (p.form == kGroupK ? p.rows : p.slot_rows);
  if (per <= (p.form == kMasked ? 64 : 32)) return kTile64x128;
  if (!fast) return per <= 128 ? kTile128x128 : kTile256x128;
  return per <= (p.form == kContiguous ? 384 : 128) ? kTile128x256 : kTile256x256;
}

// At most 16 rows, and columns that fit one launch (1024 threads for 16 of them).
bool direct_path(const BlockGemmArgs& p) {
  return p.form == kUniform && p.slot_rows <= 16 && up(p.n, 16) <= (kMaxWorkItems - 1) / 1024;
}

hipError_t launch_tiled(hipStream_t s, BlockGemmArgs p, const DeviceInfo& dev, bool fast, const Plan& pl, void* ws) {
  const BlockGemmArgs whole = p;
  if (pl.slices > 1) {
    p.slices = pl.slices;
    p.out = ws;
    p.out_kind = kOutF32;
    p.ldo = p.n;
  }
  // Results that the L2s cannot hold leave past them, and the operands stay
  // (4096x17408x5120 371 -> 357 us, FP32 K-grouped 971 -> 925 us); partial sums
  // and smaller results are read again soon.  Masked slots of at most 256 rows
  // read each weight once, by all compute units at once: those loads stream too
  // (64 slots of 256 rows, 4096x7168: 513 -> 473 us).
  const int64_t bytes = (p.form == kGroupK ? p.groups : 1) * p.rows * p.n * (p.out_kind >= kOutF32 ? 4 : 2);
  const int policy = p.form == kMasked && p.slot_rows <= 256               ? kPolStreamAll
                     : pl.slices == 1 && bytes > (int64_t)32 << 20 ? kPolStreamOut
                                                                           : kPolKeep;
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
