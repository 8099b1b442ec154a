// Token dispatch of a MoE layer: (token, slot) pairs sorted by expert, token
// rows copied (or quantised) into expert order, expert rows summed back into
// tokens with their routing weights, and that sum's gradient.
//
// A pair is i = t * topk + j with expert id ids[t, j]; ids outside [0, E) are
// unassigned.  Expert g's rows start at the previous group's end; its pairs
// take consecutive rows in the order of i, and its end is its start plus its
// count rounded up to a multiple of `align`.  Nothing here depends on the
// arrival order of atomics, so every result is the same from run to run.
#include "block_fmt.hpp"
#include "block_internal.hpp"
#include "sched.hpp"

namespace hq {
namespace {

// ------------------------------------------------------------------ sort
// A stable counting sort.  A workgroup takes a run of consecutive pairs, each
// of its waves an equal part of the run, 64 pairs a step.  A wave counts its
// pairs per expert in LDS, the counts become each wave's first row per expert,
// and the wave walks its pairs again in order: a lane's row is the wave's next
// row of its expert plus the number of lower lanes with the same expert (a
// mask built from one ballot per id bit).  A wave holds its first kHeld steps'
// ids in registers between the two walks.
// With more than one workgroup a first launch leaves every workgroup's counts
// in the workspace, and each workgroup of the second adds up what lies ahead
// of it.  The work is a few bytes a pair: launches and latency bound it, so a
// run is as short as the workgroups can cover: one step a wave up to 1024
// pairs (512 pairs of 64 experts 4.4 us; with runs of four steps 13.6), 65536
// pairs of 32 experts 4.7 + 5.9 us.
constexpr int kSortThreads = 1024, kSortWaves = kSortThreads / 64;
constexpr int kHeld = 4;
constexpr int kSortMaxBlocks = 256;

// Pairs of a workgroup's run: up to 4096 in one workgroup, else at least 2048.
int64_t sort_chunk(int64_t pairs) {
  if (pairs <= kSortThreads * kHeld) return pairs > 0 ? (pairs + kSortThreads - 1) / kSortThreads * kSortThreads : kSortThreads;
  const int64_t c = (pairs + kSortMaxBlocks - 1) / kSortMaxBlocks, least = 2 * kSortThreads;
  return ((c < least ? least : c) + kSortThreads - 1) / kSortThreads * kSortThreads;
}

__device__ __forceinline__ int pair_expert(const int64_t* ids, int64_t i, int64_t end, int E) {
  if (i >= end) return -1;
  const int64_t e = ids[i];
  return e >= 0 && e < E ? (int)e : -1;
}

__global__ __launch_bounds__(kSortThreads) void sort_count(const int64_t* __restrict__ ids, int64_t pairs, int E,
                                                           int64_t chunk, int32_t* __restrict__ ws) {
  __shared__ int cnt[kMaxGroups];
  for (int e = threadIdx.x; e < E; e += kSortThreads) cnt[e] = 0;
  __syncthreads();
  const int64_t b0 = blockIdx.x * chunk, b1 = b0 + chunk < pairs ? b0 + chunk : pairs;
  for (int64_t i = b0 + threadIdx.x; i < b1; i += kSortThreads) {
    const int e = pair_expert(ids, i, b1, E);
    if (e >= 0) atomicAdd(cnt + e, 1);
  }
  __syncthreads();
  for (int e = threadIdx.x; e < E; e += kSortThreads) ws[(int64_t)blockIdx.x * E + e] = cnt[e];
}

// Dynamic LDS: wave counts [16][E], then per expert its total, its inclusive
// padded end and the rows ahead of this workgroup.
__global__ __launch_bounds__(kSortThreads) void sort_place(const int64_t* __restrict__ ids, int64_t pairs, int E,
                                                           int align, int64_t chunk, int64_t max_rows,
                                                           const int32_t* __restrict__ ws,
                                                           int32_t* __restrict__ row_map,
                                                           int32_t* __restrict__ row_pair,
                                                           int32_t* __restrict__ group_end,
                                                           int32_t* __restrict__ counts) {
  extern __shared__ int32_t sh[];
  int32_t* wc = sh;                         // [16][E]
  int32_t* total = sh + kSortWaves * E;     // [E]
  int32_t* end = total + E;                 // [E]
  int32_t* ahead = end + E;                 // [E]
  const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6;
  const int nb = gridDim.x;
  const int64_t b0 = blockIdx.x * chunk, b1 = b0 + chunk < pairs ? b0 + chunk : pairs;
  const int64_t per = chunk / kSortWaves;
  const int64_t w0 = b0 + w * per, w1 = w0 + per < b1 ? w0 + per : b1;
  int held[kHeld];
#pragma unroll
  for (int h = 0; h < kHeld; ++h) held[h] = h * 64 < per ? pair_expert(ids, w0 + h * 64 + lane, w1, E) : -1;
  // where the counts of earlier workgroups come from: threads in parts of at
  // least E, part p adds up workgroups p, p + parts, ..
  int wide = 64;
  while (wide < E) wide <<= 1;
  int all = 0, pre = 0;
  const int parts = kSortThreads / wide, pe = tid & (wide - 1);
  if (nb > 1 && pe < E)
    for (int b = tid / wide; b < nb; b += parts) {
      const int v = ws[(int64_t)b * E + pe];
      all += v;
      pre += b < (int)blockIdx.x ? v : 0;
    }
  for (int e = tid; e < (kSortWaves + 3) * E; e += kSortThreads) sh[e] = 0;
  __syncthreads();
#pragma unroll
  for (int h = 0; h < kHeld; ++h)
    if (held[h] >= 0) atomicAdd(wc + w * E + held[h], 1);
  for (int64_t i = w0 + kHeld * 64 + lane; i < w1; i += 64) {
    const int e = pair_expert(ids, i, w1, E);
    if (e >= 0) atomicAdd(wc + w * E + e, 1);
  }
  if (nb > 1 && pe < E) {
    atomicAdd(total + pe, all);
    atomicAdd(ahead + pe, pre);
  }
  __syncthreads();
  // per expert: the waves' counts become counts before each wave
  for (int e = tid; e < E; e += kSortThreads) {
    int c[kSortWaves], s = 0;
#pragma unroll
    for (int v = 0; v < kSortWaves; ++v) c[v] = wc[v * E + e];
#pragma unroll
    for (int v = 0; v < kSortWaves; ++v) {
      wc[v * E + e] = s;
      s += c[v];
    }
    if (nb == 1) total[e] = s;
    end[e] = (total[e] + align - 1) / align * align;
  }
  __syncthreads();
  const int last = block_scan_1024<kSortThreads>(end, E, OpAdd(), 0);
  for (int e = tid; e < E; e += kSortThreads) {
    ahead[e] += e > 0 ? end[e - 1] : 0;             // the workgroup's first row of the expert
    if (blockIdx.x == 0) {
      group_end[e] = end[e];
      counts[e] = total[e];
    }
  }
  __syncthreads();
  int bits = 1;
  while ((1 << bits) < E) ++bits;
  int32_t* mine = wc + w * E;
  auto place = [&](int64_t i, int e) {
    uint64_t same = __ballot(e >= 0);
    for (int b = 0; b < bits; ++b) {
      const uint64_t m = __ballot((e >> b) & 1);
      same &= ((e >> b) & 1) ? m : ~m;
    }
    const int rank = __popcll(same & ((1ull << lane) - 1));
    int row = -1;
    if (e >= 0) row = ahead[e] + mine[e] + rank;
    __builtin_amdgcn_wave_barrier();
    if (e >= 0 && rank == 0) mine[e] += __popcll(same);
    __builtin_amdgcn_wave_barrier();
    if (i < w1) {
      row_map[i] = row;
      if (row >= 0 && row < max_rows) row_pair[row] = (int32_t)i;
    }
  };
#pragma unroll
  for (int h = 0; h < kHeld; ++h)
    if (w0 + h * 64 < w1) place(w0 + h * 64 + lane, held[h]);
  for (int64_t i0 = w0 + kHeld * 64; i0 < w1; i0 += 64) place(i0 + lane, pair_expert(ids, i0 + lane, w1, E));
  // rows that no pair takes: each group's padding, a wave a group, and what
  // follows the last end
  for (int g = blockIdx.x * kSortWaves + w; g < E; g += nb * kSortWaves) {
    const int start = (g > 0 ? end[g - 1] : 0) + total[g];
    for (int64_t r = start + lane; r < end[g] && r < max_rows; r += 64) row_pair[r] = -1;
  }
  for (int64_t r = last + (int64_t)blockIdx.x * kSortThreads + tid; r < max_rows; r += (int64_t)nb * kSortThreads)
    row_pair[r] = -1;
}

// ------------------------------------------------------------------ padding
// First padding row and end of group g, clamped to [0, max_rows].
__device__ __forceinline__ void pad_range(const PadRows& p, int g, int64_t max_rows, int64_t& r0, int64_t& r1) {
  int64_t s = g > 0 ? p.group_end[g - 1] : 0, e = p.group_end[g], c = p.counts[g];
  s = s < 0 ? 0 : s;
  c = c < 0 ? 0 : c;
  r0 = s + c;
  r1 = e < max_rows ? e : max_rows;
}

constexpr int kThreads = kMoeThreads;

// ------------------------------------------------------------------ permute
// A wave takes one 1 KB piece of one token's row, reads it once and writes it
// to each of the token's rows (16 bytes a lane): the writes bound it, and the
// reads are not repeated for each of them.  The last groups * kPadParts
// workgroups write zeros to the padding rows.
__global__ __launch_bounds__(kThreads) void permute_rows(const uint8_t* __restrict__ x, int64_t units, int64_t row_bytes,
                                                         int32_t pieces, const int32_t* __restrict__ row_map,
                                                         int32_t topk, PadRows pad, int64_t max_rows, int64_t blocks,
                                                         uint8_t* __restrict__ out) {
  typedef uint32_t v4u __attribute__((ext_vector_type(4)));
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  if ((int64_t)blockIdx.x >= blocks) {
    const int g = (int)((blockIdx.x - blocks) / kPadParts), part = (int)((blockIdx.x - blocks) % kPadParts);
    int64_t r0, r1;
    pad_range(pad, g, max_rows, r0, r1);
    for (int64_t r = r0 + part * 4 + w; r < r1; r += kPadParts * 4)
      for (int64_t c = lane; c < row_bytes / 16; c += 64)
        reinterpret_cast<v4u*>(out + r * row_bytes)[c] = v4u{0, 0, 0, 0};
    return;
  }
  const int64_t u = (int64_t)blockIdx.x * 4 + w;
  if (u >= units) return;
  const int64_t t = u / pieces, c = (u - t * pieces) * 64 + lane;
  if (c >= row_bytes / 16) return;
  const v4u v = __builtin_nontemporal_load(reinterpret_cast<const v4u*>(x + t * row_bytes) + c);
  for (int j = 0; j < topk; ++j) {
    const int32_t r = row_map[t * topk + j];
    if (r >= 0 && r < max_rows)
      __builtin_nontemporal_store(v, reinterpret_cast<v4u*>(out + (int64_t)r * row_bytes) + c);
  }
}

// The same with the row quantised to block-128 FP8 on the way: lane octets
// take 128-blocks, 16 values a lane, as the row quantiser does.  Quantised once
// a token, not once a pair.  16384 tokens top 4 of 4096 values: 75 us for 411 MB,
// 5.5 TB/s, 83 with the sort (a copy's rate would make 80).
template <bool F16>
__global__ __launch_bounds__(kThreads) void permute_quant(const uint16_t* __restrict__ x, int64_t units, int64_t h,
                                                          int32_t nkb, int32_t pieces,
                                                          const int32_t* __restrict__ row_map, int32_t topk,
                                                          PadRows pad, int64_t max_rows, int64_t blocks,
                                                          uint8_t* __restrict__ q, float* __restrict__ sf) {
  typedef uint32_t v4u __attribute__((ext_vector_type(4)));
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  if ((int64_t)blockIdx.x >= blocks) {
    const int g = (int)((blockIdx.x - blocks) / kPadParts), part = (int)((blockIdx.x - blocks) % kPadParts);
    int64_t r0, r1;
    pad_range(pad, g, max_rows, r0, r1);
    for (int64_t r = r0 + part * 4 + w; r < r1; r += kPadParts * 4) {
      for (int64_t c = lane; c < h / 16; c += 64) reinterpret_cast<v4u*>(q + r * h)[c] = v4u{0, 0, 0, 0};
      for (int64_t c = lane; c < nkb; c += 64) sf[r * nkb + c] = 0x1p-126f;
    }
    return;
  }
  const int64_t u = (int64_t)blockIdx.x * 4 + w;
  if (u >= units) return;
  const int64_t t = u / pieces;
  const int64_t c = (u - t * pieces) * 1024 + lane * 16;
  float f[16];
  uint32_t mx = 0;
  const bool in = c < h;
  if (in) {
    const uint4* p = reinterpret_cast<const uint4*>(x + t * h + c);
    const uint4 v0 = load_nt(p), v1 = load_nt(p + 1);
    unpack16<F16>(v0, v1, f);
    mx = abs_max<F16>(v0, v1);
  }
  const float s = block_scale(octet_max_u32(mx));
  if (!in) return;
  uint32_t o[4];
  block_codes(f, s, o);
  const v4u v{o[0], o[1], o[2], o[3]};
  for (int j = 0; j < topk; ++j) {
    const int32_t r = row_map[t * topk + j];
    if (r >= 0 && r < max_rows) {
      __builtin_nontemporal_store(v, reinterpret_cast<v4u*>(q + (int64_t)r * h + c));
      if ((lane & 7) == 0) sf[(int64_t)r * nkb + c / 128] = s;
    }
  }
}

// ------------------------------------------------------------------ combine
// out[t] = sum over j of weights[t, j] y[row_map[t, j]] in FP32, in slot
// order, rounded once.  A wave takes one 512-value piece of one token (16
// bytes a lane and row); the rows of four slots are loaded before they are
// added up.  The rows' bytes bound it: 1024 tokens top 8 of 2048 values 38 MB in
// 8.6 us, 4.4 TB/s, launch included.
template <bool F16>
__global__ __launch_bounds__(kThreads) void combine_rows(const uint16_t* __restrict__ y, int64_t units, int64_t h,
                                                         int32_t pieces, const int32_t* __restrict__ row_map,
                                                         int32_t topk, const float* __restrict__ weights,
                                                         int64_t max_rows, uint16_t* __restrict__ out) {
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  const int64_t u = (int64_t)blockIdx.x * 4 + w;
  if (u >= units) return;
  const int64_t t = u / pieces, c = (u - t * pieces) * 512 + lane * 8;
  if (c >= h) return;
  float acc[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) acc[i] = 0.0f;
  for (int j0 = 0; j0 < topk; j0 += 4) {
    uint4 v[4];
    float wt[4];
    bool on[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      on[j] = false;
      if (j0 + j < topk) {
        const int32_t r = row_map[t * topk + j0 + j];
        on[j] = r >= 0 && r < max_rows;
        if (on[j]) {
          wt[j] = weights != nullptr ? weights[t * topk + j0 + j] : 1.0f;
          v[j] = load_nt(reinterpret_cast<const uint4*>(y + (int64_t)r * h + c));
        }
      }
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (!on[j]) continue;
      const uint32_t d[4] = {v[j].x, v[j].y, v[j].z, v[j].w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        acc[2 * i] = __builtin_fmaf(wt[j], half_lo<F16>(d[i]), acc[2 * i]);
        acc[2 * i + 1] = __builtin_fmaf(wt[j], half_hi<F16>(d[i]), acc[2 * i + 1]);
      }
    }
  }
  uint4 o;
  o.x = pack_half2<F16>(acc[0], acc[1]);
  o.y = pack_half2<F16>(acc[2], acc[3]);
  o.z = pack_half2<F16>(acc[4], acc[5]);
  o.w = pack_half2<F16>(acc[6], acc[7]);
  *reinterpret_cast<uint4*>(out + t * h + c) = o;
}

// dy[row] = weights[t, j] dout[t] and dweights[t, j] = dout[t] . y[row], the
// product summed in FP32.  One workgroup takes a token, each of its waves (up
// to eight) a slot at a time: a lane's share of the row, 16 bytes of every
// kilobyte, four loads in flight, then one reduction over the wave in a fixed
// order.  dout's row comes from memory once and from a cache for the other
// waves.  The bytes of y and dy bound it; with few tokens the chain of loads
// behind a slot does, and a wave a slot keeps that chain one row long.  16384
// tokens top 4 of 4096 values: 1.21 GB in 204 to 224 us, 5.4 to 5.9 TB/s.
template <bool F16, bool NT>
__global__ __launch_bounds__(512) void combine_bwd(const uint16_t* __restrict__ dout, const uint16_t* __restrict__ y,
                                                   int64_t tokens, int64_t h, const int32_t* __restrict__ row_map,
                                                   int32_t topk, const float* __restrict__ weights, PadRows pad,
                                                   int64_t max_rows, uint16_t* __restrict__ dy,
                                                   float* __restrict__ dweights) {
  const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6, waves = blockDim.x >> 6;
  const int64_t chunks = h / 8;
  if ((int64_t)blockIdx.x >= tokens) {
    const int g = (int)((blockIdx.x - tokens) / kPadParts), p = (int)((blockIdx.x - tokens) % kPadParts);
    int64_t r0, r1;
    pad_range(pad, g, max_rows, r0, r1);
    for (int64_t r = r0 + p * waves + w; r < r1; r += kPadParts * waves)
      for (int64_t c = lane; c < chunks; c += 64) store16<NT>(dy + r * h + 8 * c, u32x4{0, 0, 0, 0});
    return;
  }
  const int64_t t = blockIdx.x;
  const uint4* dt = reinterpret_cast<const uint4*>(dout + t * h);
  for (int j = w; j < topk; j += waves) {
    const int32_t r = row_map[t * topk + j];
    float dot = 0.0f;
    if (r >= 0 && r < max_rows) {
      const float wt = weights[t * topk + j];
      const uint4* yr = reinterpret_cast<const uint4*>(y + (int64_t)r * h);
      uint16_t* out = dy + (int64_t)r * h;
      for (int64_t c0 = lane; c0 < chunks; c0 += 256) {
        uint4 dv[4], yv[4];
#pragma unroll
        for (int u = 0; u < 4; ++u)
          if (c0 + 64 * u < chunks) {
            dv[u] = dt[c0 + 64 * u];
            yv[u] = load_nt(yr + c0 + 64 * u);
          }
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          if (c0 + 64 * u >= chunks) continue;
          const uint32_t d[4] = {dv[u].x, dv[u].y, dv[u].z, dv[u].w}, v[4] = {yv[u].x, yv[u].y, yv[u].z, yv[u].w};
          u32x4 o;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float a = half_lo<F16>(d[i]), b = half_hi<F16>(d[i]);
            dot = __builtin_fmaf(a, half_lo<F16>(v[i]), dot);
            dot = __builtin_fmaf(b, half_hi<F16>(v[i]), dot);
            o[i] = pack_half2<F16>(wt * a, wt * b);
          }
          store16<NT>(out + 8 * (c0 + 64 * u), o);
        }
      }
      for (int off = 32; off >= 1; off >>= 1) dot += __shfl_xor(dot, off, 64);
    }
    if (lane == 0) dweights[t * topk + j] = dot;
  }
}

}  // namespace

uint64_t moe_sort_workspace_bytes(int64_t pairs, int32_t experts) {
  const int64_t chunk = sort_chunk(pairs), nb = (pairs + chunk - 1) / chunk;
  return nb > 1 ? (uint64_t)(nb * experts) * sizeof(int32_t) : 0;
}

hipError_t launch_moe_sort(hipStream_t s, const int64_t* ids, int64_t pairs, int32_t experts, int32_t align,
                           int64_t max_rows, int32_t* row_map, int32_t* row_pair, int32_t* group_end,
                           int32_t* counts, void* workspace) {
  const int64_t chunk = sort_chunk(pairs);
  int64_t nb = (pairs + chunk - 1) / chunk;
  nb = nb < 1 ? 1 : nb;
  int32_t* ws = static_cast<int32_t*>(workspace);
  if (nb > 1) {
    hipLaunchKernelGGL(sort_count, dim3((unsigned)nb), dim3(kSortThreads), 0, s, ids, pairs, experts, chunk, ws);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  const size_t lds = sizeof(int32_t) * (size_t)(kSortWaves + 3) * experts;
  if (lds > 65536) {
    const hipError_t e = hipFuncSetAttribute((const void*)sort_place, hipFuncAttributeMaxDynamicSharedMemorySize,
                                             (int)(sizeof(int32_t) * (kSortWaves + 3) * kMaxGroups));
    if (e != hipSuccess) return e;
  }
  hipLaunchKernelGGL(sort_place, dim3((unsigned)nb), dim3(kSortThreads), lds, s, ids, pairs, experts, align, chunk,
                     max_rows, (const int32_t*)ws, row_map, row_pair, group_end, counts);
  return hipGetLastError();
}

hipError_t launch_moe_permute(hipStream_t s, const uint8_t* x, int64_t tokens, int64_t row_bytes,
                              const int32_t* row_map, int32_t topk, PadRows pad, int64_t max_rows, uint8_t* out) {
  const int64_t pieces = (row_bytes + 1023) / 1024, units = tokens * pieces;
  const int64_t blocks = piece_groups(tokens, row_bytes, 1024);
  if (blocks + pad_groups(pad) == 0) return hipSuccess;
  hipLaunchKernelGGL(permute_rows, dim3((unsigned)(blocks + pad_groups(pad))), dim3(kThreads), 0, s, x, units,
                     row_bytes, (int32_t)pieces, row_map, topk, pad, max_rows, blocks, out);
  return hipGetLastError();
}

hipError_t launch_moe_permute_block_quant(hipStream_t s, const uint16_t* x, int64_t tokens, int64_t h,
                                          const int32_t* row_map, int32_t topk, PadRows pad, int64_t max_rows,
                                          uint8_t* q, float* sf, bool fp16) {
  const int64_t pieces = (h + 1023) / 1024, units = tokens * pieces, blocks = piece_groups(tokens, h, 1024);
  if (blocks + pad_groups(pad) == 0) return hipSuccess;
  const dim3 grid((unsigned)(blocks + pad_groups(pad)));
  const int32_t nkb = (int32_t)((h + 127) / 128);
  if (fp16)
    hipLaunchKernelGGL(permute_quant<true>, grid, dim3(kThreads), 0, s, x, units, h, nkb, (int32_t)pieces, row_map, topk,
                       pad, max_rows, blocks, q, sf);
  else
    hipLaunchKernelGGL(permute_quant<false>, grid, dim3(kThreads), 0, s, x, units, h, nkb, (int32_t)pieces, row_map,
                       topk, pad, max_rows, blocks, q, sf);
  return hipGetLastError();
}

hipError_t launch_moe_combine(hipStream_t s, const uint16_t* y, int64_t tokens, int64_t h, const int32_t* row_map,
                              int32_t topk, const float* weights, int64_t max_rows, uint16_t* out, bool fp16) {
  const int64_t pieces = (h + 511) / 512, units = tokens * pieces;
  const dim3 grid((unsigned)piece_groups(tokens, h, 512));
  if (fp16)
    hipLaunchKernelGGL(combine_rows<true>, grid, dim3(kThreads), 0, s, y, units, h, (int32_t)pieces, row_map, topk,
                       weights, max_rows, out);
  else
    hipLaunchKernelGGL(combine_rows<false>, grid, dim3(kThreads), 0, s, y, units, h, (int32_t)pieces, row_map, topk,
                       weights, max_rows, out);
  return hipGetLastError();
}

hipError_t launch_moe_combine_backward(hipStream_t s, const uint16_t* dout, const uint16_t* y, int64_t tokens,
                                       int64_t h, const int32_t* row_map, int32_t topk, const float* weights,
                                       PadRows pad, int64_t max_rows, uint16_t* dy, float* dweights, bool fp16) {
  const int64_t blocks = tokens + pad_groups(pad);
  if (blocks == 0) return hipSuccess;
  const int waves = combine_bwd_waves(topk);
  const bool nt = max_rows * h * 2 > kStreamBytes;
#define HQ_BWD(F, N)                                                                                               \
  hipLaunchKernelGGL((combine_bwd<F, N>), dim3((unsigned)blocks), dim3(64 * waves), 0, s, dout, y, tokens, h, row_map, \
                     topk, weights, pad, max_rows, dy, dweights)
  if (fp16 && nt) HQ_BWD(true, true);
  else if (fp16) HQ_BWD(true, false);
  else if (nt) HQ_BWD(false, true);
  else HQ_BWD(false, false);
#undef HQ_BWD
  return hipGetLastError();
}

}  // namespace hq
