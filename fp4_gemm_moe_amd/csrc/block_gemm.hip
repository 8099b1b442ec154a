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
// A workgroup of W waves takes 16 MF rows x 16 NF columns; its waves take the
// K blocks in turn, each lane loading its operands from global memory, and
// their sums meet in LDS.
template <int MF, int NF, int W>
__global__ __launch_bounds__(W * 64) void block_gemm_direct(BlockGemmArgs p) {
  __shared__ int ends[kMaxGroups];
  __shared__ v4f part[W > 1 ? W - 1 : 1][MF * NF][64];
  const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6;
  const int r16 = lane & 15, q = lane >> 4;
  const int g = blockIdx.y;
  int64_t row0 = 0, row_end = p.rows;
  int kb0 = 0, kb1 = p.nkb;
  if (p.form == kContiguous || p.form == kGroupK) {
    load_clamped_ends<W * 64>(ends, p.group_end, p.groups, p.form == kContiguous ? p.rows : p.k);
    const int lo = g > 0 ? ends[g - 1] : 0, hi = ends[g];
    if (p.form == kContiguous) {
      row0 = lo;
      row_end = hi;
    } else {
      kb0 = lo / 128;
      kb1 = hi / 128;
    }
  } else {
    row0 = g * p.slot_rows;
    int64_t c = p.slot_rows;
    if (p.form == kMasked) {
      c = p.counts[g];
      c = c < 0 ? 0 : (c > p.slot_rows ? p.slot_rows : c);
    }
    row_end = row0 + c;
  }
  const int64_t n0 = (int64_t)blockIdx.x * 16 * NF;
  const bool own_b = p.form != kGroupK;
  const uint8_t* b = p.b + (own_b ? (int64_t)g * p.n * p.k : 0);
  const float* sb = p.sb + (own_b ? (int64_t)g * p.nnb * p.nkb : 0) + (n0 / 128) * p.nkb;
  const uint8_t* bp[NF];
#pragma unroll
  for (int j = 0; j < NF; ++j) {
    const int64_t n = n0 + 16 * j + r16;
    bp[j] = b + (n < p.n ? n : p.n - 1) * p.k;
  }
  for (int64_t m0 = row0 + (int64_t)blockIdx.z * 16 * MF; m0 < row_end; m0 += (int64_t)gridDim.z * 16 * MF) {
    const uint8_t* ap[MF];
    const float* sap[MF];
#pragma unroll
    for (int i = 0; i < MF; ++i) {
      const int64_t r = m0 + 16 * i + r16;
      ap[i] = p.a + (r < row_end ? r : row_end - 1) * p.k;
      sap[i] = p.sa + (r < row_end ? r : row_end - 1) * p.nkb;
    }
    v4f acc[MF][NF];
#pragma unroll
    for (int i = 0; i < MF; ++i)
#pragma unroll
      for (int j = 0; j < NF; ++j) acc[i][j] = v4f{0, 0, 0, 0};
    for (int kb = kb0 + w; kb < kb1; kb += W) {
      const int64_t k0 = (int64_t)kb * 128 + 16 * q;
      const bool in0 = k0 < p.k, in1 = k0 + 64 < p.k;
      v8i bf[NF];
#pragma unroll
      for (int j = 0; j < NF; ++j) bf[j] = load_pair(bp[j] + k0, in0, in1);
      const float sbv = sb[kb];
#pragma unroll
      for (int i = 0; i < MF; ++i) {
        const v8i af = load_pair(ap[i] + k0, in0, in1);
        const float f = sap[i][kb] * sbv;
#pragma unroll
        for (int j = 0; j < NF; ++j) {
          const v4f t = dot16(bf[j], af);
#pragma unroll
          for (int e = 0; e < 4; ++e) acc[i][j][e] = __builtin_fmaf(t[e], f, acc[i][j][e]);
        }
      }
    }
    if (W > 1) {
      __syncthreads();
      if (w > 0)
#pragma unroll
        for (int i = 0; i < MF; ++i)
#pragma unroll
          for (int j = 0; j < NF; ++j) part[w - 1][i * NF + j][lane] = acc[i][j];
      __syncthreads();
    }
    if (w == 0) {
#pragma unroll
      for (int i = 0; i < MF; ++i)
#pragma unroll
        for (int j = 0; j < NF; ++j) {
          v4f v = acc[i][j];
          for (int o = 0; o < W - 1; ++o) v += part[o][i * NF + j][lane];
          const int64_t r = m0 + 16 * i + r16, n = n0 + 16 * j + 4 * q;
          if (r < row_end && n < p.n)
            store4(p.out, p.out_kind, ((p.form == kGroupK ? (int64_t)g * p.rows : 0) + r) * p.n + n, v);
        }
    }
  }
}

// ------------------------------------------------------------------ K split
// out = the slices' FP32 partial sums, added in slice order.
constexpr int kReduceThreads = 256;
__global__ __launch_bounds__(kReduceThreads) void block_reduce(const float* __restrict__ partial, int slices,
                                                               int64_t quads, void* out, int32_t kind) {
  const int64_t i = (int64_t)blockIdx.x * kReduceThreads + threadIdx.x;
  if (i >= quads) return;
  const v4f* src = reinterpret_cast<const v4f*>(partial) + i;
  v4f v = src[0];
  for (int s = 1; s < slices; ++s) v += src[s * quads];
  store4(out, kind, 4 * i, v);
}

bool fast_path(const BlockGemmArgs& p) { return p.out_kind == kOutBf16 && p.nkb >= 4; }

struct Plan {
  bool direct;
  int tile;
  int slices;
  uint64_t bytes;      // workspace of the split
};

Plan plan_gemm(const BlockGemmArgs& p, const DeviceInfo& dev) {
  Plan pl{false, kTile256x256, 1, 0};
  const bool fast = fast_path(p);
  const int64_t per = p.form == kContiguous ? (p.rows + p.groups - 1) / p.groups
                                            : (p.form == kGroupK ? p.rows : p.slot_rows);
  if (p.form == kUniform && p.slot_rows <= 16) {
    pl.direct = true;
    return pl;
  }
  int bm = 256, bn = 256;
  if (per <= 64 || p.nkb < 4) {        // the larger tiles fetch four K blocks' scales at a time
    pl.tile = kTile64x128;
    bm = 64, bn = 128;
  } else if (fast && per <= 128) {
    pl.tile = kTile128x128;
    bm = 128, bn = 128;
  } else if (!fast) {
    pl.tile = kTile256x128;
    bn = 128;
  }
  if (p.form == kUniform) {
    const int64_t tiles = (p.slot_rows + bm - 1) / bm * p.groups * ((p.n + bn - 1) / bn);
    int64_t s = dev.num_cus / tiles;
    if (s > p.nkb / 4) s = p.nkb / 4;
    const int64_t most = (int64_t)(HQ_BLOCK_WORKSPACE_BYTES / 4) / (p.rows * p.n);
    if (s > most) s = most;
    if (s > 1) {
      pl.slices = (int)s;
      pl.bytes = (uint64_t)s * p.rows * p.n * 4;
    }
  }
  return pl;
}

}  // namespace

uint64_t block_gemm_workspace_bytes(const BlockGemmArgs& p, const DeviceInfo& dev) { return plan_gemm(p, dev).bytes; }

hipError_t launch_block_gemm(hipStream_t s, const BlockGemmArgs& args, const DeviceInfo& dev, void* workspace,
                             uint64_t workspace_bytes) {
  const Plan pl = plan_gemm(args, dev);
  BlockGemmArgs p = args;
  if (pl.direct) {
    constexpr int MF = 1, NF = 1, W = 8;
    const dim3 grid((unsigned)((p.n + 16 * NF - 1) / (16 * NF)), (unsigned)p.groups, 1);
    hipLaunchKernelGGL((block_gemm_direct<MF, NF, W>), grid, dim3(W * 64), 0, s, p);
    return hipGetLastError();
  }
  const bool nt = p.form == kMasked && p.slot_rows <= 256;
  const bool split = pl.slices > 1 && workspace_bytes >= pl.bytes;
  if (split) {
    p.slices = pl.slices;
    p.out = workspace;
    p.out_kind = kOutF32;
  }
  hipError_t e = fast_path(args) ? launch_block_fast(s, p, dev, pl.tile, nt) : launch_block_exact(s, p, dev, pl.tile, nt);
  if (e != hipSuccess || !split) return e;
  const int64_t quads = p.rows * p.n / 4;
  hipLaunchKernelGGL(block_reduce, dim3((unsigned)((quads + kReduceThreads - 1) / kReduceThreads)), dim3(kReduceThreads),
                     0, s, static_cast<const float*>(workspace), pl.slices, quads, args.out, args.out_kind);
  return hipGetLastError();
}

}  // namespace hq
