// A plain 64 x 64 tile of a product summed in FP32 by vector instructions: a
// workgroup of 256 threads, four rows and four columns a thread.
#pragma once

#include "block_fmt.hpp"
#include "sched.hpp"

namespace hq {

template <bool F16>
__device__ __forceinline__ float half_value(uint16_t v) {
  if constexpr (F16) return f16_lo(v);
  else return bf16_lo(v);
}
template <bool F16>
__device__ __forceinline__ uint16_t to_half(float v) {
  return (uint16_t)pack_half2<F16>(v, 0.0f);
}

// sum over kk < K of la(i, kk) lb(j, kk), given to st(i, j, sum) for i, j < 64.
template <class LA, class LB, class ST>
__device__ __forceinline__ void plain_tile(int64_t K, LA la, LB lb, ST st) {
  __shared__ float a[16][65], b[16][65];
  const int t = threadIdx.x, ti = t >> 4, tj = t & 15;
  float acc[4][4] = {};
  for (int64_t k0 = 0; k0 < K; k0 += 16) {
    for (int e = t; e < 1024; e += 256) {
      const int i = e >> 4, kk = e & 15;
      a[kk][i] = k0 + kk < K ? la(i, k0 + kk) : 0.0f;
      b[kk][i] = k0 + kk < K ? lb(i, k0 + kk) : 0.0f;
    }
    __syncthreads();
    for (int kk = 0; kk < 16; ++kk)
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = __builtin_fmaf(a[kk][ti * 4 + i], b[kk][tj * 4 + j], acc[i][j]);
    __syncthreads();
  }
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) st(ti * 4 + i, tj * 4 + j, acc[i][j]);
}

// The group and first row of m-tile mt (64 rows) over groups that end at
// ends[g]; g == groups where there is none.
struct PlainTile {
  int g;
  int64_t row0, row_end;
};
__device__ __forceinline__ PlainTile plain_find(const int* ends, int groups, int mt) {
  int start = 0;
  for (int g = 0; g < groups; ++g) {
    const int tiles = (ends[g] - start + 63) / 64;
    if (mt < tiles) return {g, start + (int64_t)mt * 64, ends[g]};
    mt -= tiles;
    start = ends[g];
  }
  return {groups, 0, 0};
}

}  // namespace hq
