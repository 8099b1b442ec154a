// 16-bit products by expert: out[r] = a[r] b[g]^T (or a[r] b[g]) for the rows r
// of group g, and out[g] = sum over its rows of a[r]^T b[r].
#include "half_internal.hpp"
#include "half_plain.hpp"

namespace hq {
namespace {

__device__ __forceinline__ void store_out(void* out, int32_t kind, int64_t at, float v) {
  if (kind == kOutBf16) static_cast<uint16_t*>(out)[at] = to_half<false>(v);
  else if (kind == kOutF16) static_cast<uint16_t*>(out)[at] = to_half<true>(v);
  else if (kind == kOutF32) static_cast<float*>(out)[at] = v;
  else static_cast<float*>(out)[at] += v;
}

template <bool F16>
__global__ __launch_bounds__(256) void half_plain_kernel(HalfGemmArgs p) {
  __shared__ int ends[kMaxGroups];
  const int nt = (int)((p.n + 63) / 64);
  int id = blockIdx.x;
  const int64_t n0 = (int64_t)(id % nt) * 64;
  id /= nt;
  if (p.form == kGroupK) {
    load_clamped_ends<256>(ends, p.group_end, p.groups, p.k);
    const int mt = (int)((p.rows + 63) / 64), g = id / mt;
    const int64_t m0 = (int64_t)(id % mt) * 64, lo = g > 0 ? ends[g - 1] : 0;
    plain_tile(
        ends[g] - lo, [&](int i, int64_t kk) { return m0 + i < p.rows ? half_value<F16>(p.a[(lo + kk) * p.rows + m0 + i]) : 0.0f; },
        [&](int j, int64_t kk) { return n0 + j < p.n ? half_value<F16>(p.b[(lo + kk) * p.n + n0 + j]) : 0.0f; },
        [&](int i, int j, float v) {
          if (m0 + i < p.rows && n0 + j < p.n) store_out(p.out, p.out_kind, (g * p.rows + m0 + i) * p.n + n0 + j, v);
        });
    return;
  }
  PlainTile t;
  if (p.form == kContiguous) {
    load_clamped_ends<256>(ends, p.group_end, p.groups, p.rows);
    t = plain_find(ends, p.groups, id);
    if (t.g >= p.groups) return;
  } else {
    const int mt = (int)((p.slot_rows + 63) / 64);
    t.g = id / mt;
    int64_t c = p.counts[t.g];
    c = c < 0 ? 0 : (c > p.slot_rows ? p.slot_rows : c);
    t.row0 = t.g * p.slot_rows + (int64_t)(id % mt) * 64;
    t.row_end = t.g * p.slot_rows + c;
    if (t.row0 >= t.row_end) return;
  }
  const uint16_t* b = p.b + (int64_t)t.g * p.n * p.k;
  plain_tile(
      p.k, [&](int i, int64_t kk) { return t.row0 + i < t.row_end ? half_value<F16>(p.a[(t.row0 + i) * p.k + kk]) : 0.0f; },
      [&](int j, int64_t kk) {
        return n0 + j < p.n ? half_value<F16>(p.b_t ? b[kk * p.n + n0 + j] : b[(n0 + j) * p.k + kk]) : 0.0f;
      },
      [&](int i, int j, float v) {
        if (t.row0 + i < t.row_end && n0 + j < p.n) store_out(p.out, p.out_kind, (t.row0 + i) * p.n + n0 + j, v);
      });
}

}  // namespace

hipError_t launch_half_gemm(hipStream_t s, const HalfGemmArgs& p, const DeviceInfo&) {
  const int64_t nt = (p.n + 63) / 64;
  int64_t tiles = p.form == kContiguous ? (p.rows / 64 + p.groups) * nt
                  : p.form == kMasked   ? (p.slot_rows + 63) / 64 * p.groups * nt
                                        : (p.rows + 63) / 64 * p.groups * nt;
  if (p.f16) hipLaunchKernelGGL(half_plain_kernel<true>, dim3((unsigned)tiles), dim3(256), 0, s, p);
  else hipLaunchKernelGGL(half_plain_kernel<false>, dim3((unsigned)tiles), dim3(256), 0, s, p);
  return hipGetLastError();
}

}  // namespace hq
