// Low-rank adapters: v = x A[g]^T by place, out = base + scale[g] v B[g]^T by
// token, and the gradients dx, dA, dB.
#include "half_internal.hpp"
#include "half_plain.hpp"

namespace hq {
namespace {

__device__ __forceinline__ int64_t token_at(const LoraPlan& pl, int64_t place) {
  const int64_t t = pl.row_pair != nullptr ? pl.row_pair[place] : place;
  return t >= 0 && t < pl.m ? t : -1;
}

// out[place, r] = z[token] w[g]^T, w [r, k] (t: [k, r])
template <bool F16>
__global__ __launch_bounds__(256) void shrink_kernel(LoraPlan pl, const uint16_t* z, const uint16_t* w, bool t,
                                                     int64_t k, int64_t r, float* out) {
  __shared__ int ends[kMaxGroups];
  const int nt = (int)((r + 63) / 64);
  const int64_t n0 = (int64_t)(blockIdx.x % nt) * 64;
  load_clamped_ends<256>(ends, pl.group_end, pl.adapters, pl.max_rows);
  const PlainTile tl = plain_find(ends, pl.adapters, blockIdx.x / nt);
  if (tl.g >= pl.adapters) return;
  w += (int64_t)tl.g * r * k;
  plain_tile(
      k,
      [&](int i, int64_t kk) {
        const int64_t tok = tl.row0 + i < tl.row_end ? token_at(pl, tl.row0 + i) : -1;
        return tok >= 0 ? half_value<F16>(z[tok * k + kk]) : 0.0f;
      },
      [&](int j, int64_t kk) { return n0 + j < r ? half_value<F16>(t ? w[kk * r + n0 + j] : w[(n0 + j) * k + kk]) : 0.0f; },
      [&](int i, int j, float v) {
        if (tl.row0 + i < tl.row_end && n0 + j < r && token_at(pl, tl.row0 + i) >= 0) out[(tl.row0 + i) * r + n0 + j] = v;
      });
}

// out[token, n] = base + scale v[place] w[g]^T, w [n, r] (t: [r, n])
template <bool F16>
__global__ __launch_bounds__(256) void expand_kernel(LoraPlan pl, const float* v, const uint16_t* w, bool t,
                                                     const uint16_t* base, uint16_t* out, int64_t n, int64_t r) {
  __shared__ int ends[kMaxGroups];
  const int nt = (int)((n + 63) / 64);
  const int64_t n0 = (int64_t)(blockIdx.x % nt) * 64;
  load_clamped_ends<256>(ends, pl.group_end, pl.adapters, pl.max_rows);
  const PlainTile tl = plain_find(ends, pl.adapters, blockIdx.x / nt);
  if (tl.g >= pl.adapters) return;
  w += (int64_t)tl.g * r * n;
  const float f = pl.scale != nullptr ? pl.scale[tl.g] : 1.0f;
  plain_tile(
      r,
      [&](int i, int64_t kk) {
        return tl.row0 + i < tl.row_end && token_at(pl, tl.row0 + i) >= 0 ? v[(tl.row0 + i) * r + kk] : 0.0f;
      },
      [&](int j, int64_t kk) { return n0 + j < n ? half_value<F16>(t ? w[kk * n + n0 + j] : w[(n0 + j) * r + kk]) : 0.0f; },
      [&](int i, int j, float s) {
        const int64_t tok = tl.row0 + i < tl.row_end && n0 + j < n ? token_at(pl, tl.row0 + i) : -1;
        if (tok < 0) return;
        const int64_t at = tok * n + n0 + j;
        out[at] = to_half<F16>((base != nullptr ? half_value<F16>(base[at]) : 0.0f) + f * s);
      });
}

// Rows of tokens without an adapter: base, or zeros.
__global__ __launch_bounds__(256) void rest_kernel(LoraPlan pl, const uint16_t* base, uint16_t* out, int64_t n) {
  __shared__ int ends[kMaxGroups];
  load_clamped_ends<256>(ends, pl.group_end, pl.adapters, pl.max_rows);
  const int64_t t = blockIdx.x;
  const int64_t place = pl.row_map != nullptr ? pl.row_map[t] : t;
  if (place >= 0 && place < ends[pl.adapters - 1]) return;
  for (int64_t c = threadIdx.x; c < n; c += 256) out[t * n + c] = base != nullptr ? base[t * n + c] : 0;
}

// da[g, i, j] = scale sum over places of u[place, i] z[token, j]; t: stored as [j, i]
template <bool F16>
__global__ __launch_bounds__(256) void outer_kernel(LoraPlan pl, const float* u, const uint16_t* z, int64_t r, int64_t k,
                                                    bool t, bool accumulate, float* out) {
  __shared__ int ends[kMaxGroups];
  const int kt = (int)((k + 63) / 64), rt = (int)((r + 63) / 64);
  int id = blockIdx.x;
  const int64_t k0 = (int64_t)(id % kt) * 64;
  id /= kt;
  const int64_t r0 = (int64_t)(id % rt) * 64;
  const int g = id / rt;
  load_clamped_ends<256>(ends, pl.group_end, pl.adapters, pl.max_rows);
  const int64_t lo = g > 0 ? ends[g - 1] : 0;
  const float f = pl.scale != nullptr ? pl.scale[g] : 1.0f;
  plain_tile(
      ends[g] - lo,
      [&](int i, int64_t kk) { return r0 + i < r && token_at(pl, lo + kk) >= 0 ? u[(lo + kk) * r + r0 + i] : 0.0f; },
      [&](int j, int64_t kk) {
        const int64_t tok = k0 + j < k ? token_at(pl, lo + kk) : -1;
        return tok >= 0 ? half_value<F16>(z[tok * k + k0 + j]) : 0.0f;
      },
      [&](int i, int j, float s) {
        if (r0 + i >= r || k0 + j >= k) return;
        float* o = out + g * r * k + (t ? (k0 + j) * r + r0 + i : (r0 + i) * k + k0 + j);
        *o = f * s + (accumulate ? *o : 0.0f);
      });
}

unsigned tiles(const LoraPlan& pl, int64_t n) {
  return (unsigned)((pl.max_rows / 64 + pl.adapters) * ((n + 63) / 64));
}

template <bool F16>
hipError_t forward(hipStream_t s, const LoraArgs& p) {
  float* v = p.v != nullptr ? p.v : static_cast<float*>(p.workspace);
  hipLaunchKernelGGL(shrink_kernel<F16>, dim3(tiles(p.plan, p.r)), dim3(256), 0, s, p.plan, p.x, p.a, false, p.k, p.r, v);
  hipLaunchKernelGGL(expand_kernel<F16>, dim3(tiles(p.plan, p.n)), dim3(256), 0, s, p.plan, v, p.b, false, p.base, p.out,
                     p.n, p.r);
  if (p.base != p.out)
    hipLaunchKernelGGL(rest_kernel, dim3((unsigned)p.plan.m), dim3(256), 0, s, p.plan, p.base, p.out, p.n);
  return hipGetLastError();
}

template <bool F16>
hipError_t backward(hipStream_t s, const LoraArgs& p) {
  float* u = static_cast<float*>(p.workspace);
  const LoraPlan& pl = p.plan;
  hipLaunchKernelGGL(shrink_kernel<F16>, dim3(tiles(pl, p.r)), dim3(256), 0, s, pl, p.dy, p.b, true, p.n, p.r, u);
  if (p.out != nullptr) {
    hipLaunchKernelGGL(expand_kernel<F16>, dim3(tiles(pl, p.k)), dim3(256), 0, s, pl, u, p.a, true, p.base, p.out, p.k,
                       p.r);
    if (p.base != p.out && pl.m > 0)
      hipLaunchKernelGGL(rest_kernel, dim3((unsigned)pl.m), dim3(256), 0, s, pl, p.base, p.out, p.k);
  }
  const int64_t rt = (p.r + 63) / 64;
  hipLaunchKernelGGL(outer_kernel<F16>, dim3((unsigned)(rt * ((p.k + 63) / 64) * pl.adapters)), dim3(256), 0, s, pl, u,
                     p.x, p.r, p.k, false, p.accumulate, p.da);
  hipLaunchKernelGGL(outer_kernel<F16>, dim3((unsigned)(rt * ((p.n + 63) / 64) * pl.adapters)), dim3(256), 0, s, pl, p.v,
                     p.dy, p.r, p.n, true, p.accumulate, p.db);
  return hipGetLastError();
}

}  // namespace

uint64_t lora_workspace_bytes(int64_t max_rows, int64_t, int64_t, int64_t r, int32_t) { return (uint64_t)max_rows * r * 4; }
uint64_t lora_backward_workspace_bytes(int64_t max_rows, int64_t, int64_t, int64_t r, int32_t) {
  return (uint64_t)max_rows * r * 4;
}

hipError_t launch_lora(hipStream_t s, const LoraArgs& p) { return p.f16 ? forward<true>(s, p) : forward<false>(s, p); }
hipError_t launch_lora_backward(hipStream_t s, const LoraArgs& p) {
  return p.f16 ? backward<true>(s, p) : backward<false>(s, p);
}

}  // namespace hq
