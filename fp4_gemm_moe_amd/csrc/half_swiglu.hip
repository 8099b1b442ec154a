// SwiGLU in 16 bits and its gradient: x = [gate | up] (rows of 2h values),
//   s = 1 / (1 + exp(-gate)),  y = up gate s,
//   dgate = dy up s (1 + gate (1 - s)),  dup = dy gate s
// in FP32, each result rounded once.  With t = exp(-|gate|), which cannot
// overflow, s and 1 - s are 1 / (1 + t) and t / (1 + t) in the order of the
// gate's sign, so neither loses digits to the other.
//
// Memory bounds both: 6 bytes move for each y, 10 for each y of the gradient, 12
// where it writes y too.  A thread takes eight neighbouring values of a row, in
// 16-byte words: 65536 x 1536 with y 213 us, 5.67 TB/s (a copy of 256 MB 5.4); 512 x
// 2048 3.2 us, one launch's latency.  By group every workgroup scans the ends before
// its rows are read: 65536 x 1536 103 us for all rows, 104 in 32 slots, 122 by 32 ends
// and 128 by 256; the gradient 212, 212 and 214 (32 ends).
#include "block_fmt.hpp"
#include "half_internal.hpp"
#include "sched.hpp"

namespace hq {
namespace {

constexpr int kThreads = 256;

struct Sig {
  float s, not_s;      // sigmoid(gate), 1 - sigmoid(gate)
};
__device__ __forceinline__ Sig sigmoid(float gate) {
  const float t = __builtin_amdgcn_exp2f(__builtin_fabsf(gate) * -1.4426950408889634f);
  const float r = __builtin_amdgcn_rcpf(1.0f + t), tr = t * r;
  return gate >= 0.0f ? Sig{r, tr} : Sig{tr, gate < 0.0f ? r : gate};      // a NaN gate stays one
}

template <bool F16>
__device__ __forceinline__ void unpack8(const u32x4& u, float (&f)[8]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = half_lo<F16>(u[i]);
    f[2 * i + 1] = half_hi<F16>(u[i]);
  }
}
template <bool F16>
__device__ __forceinline__ u32x4 pack8(const float (&f)[8]) {
  return u32x4{pack_half2<F16>(f[0], f[1]), pack_half2<F16>(f[2], f[3]), pack_half2<F16>(f[4], f[5]),
               pack_half2<F16>(f[6], f[7])};
}

// Is row r selected?
__device__ __forceinline__ bool selected(const RowSelection& sel, const int* ends, uint32_t r) {
  if (sel.groups == 0) return true;
  int64_t start, g;
  if (sel.group_end != nullptr) {
    g = find_group(ends, sel.groups, (int)r);
    if (g >= sel.groups) return false;
    start = g > 0 ? ends[g - 1] : 0;
  } else {
    g = r / sel.slot_rows;
    if (g >= sel.groups) return false;
    start = g * sel.slot_rows;
  }
  return sel.valid == nullptr || (int64_t)r - start < sel.valid[g];
}

// BWD: dy and dx are given, y may be.
template <bool F16, bool BWD>
__global__ __launch_bounds__(kThreads) void swiglu_kernel(const u32x4* dy, const u32x4* x, uint32_t rows, uint32_t nch,
                                                          RowSelection sel, u32x4* dx, u32x4* y) {
  __shared__ int ends[kMaxGroups];
  if (sel.group_end != nullptr) load_clamped_ends<kThreads>(ends, sel.group_end, sel.groups, rows);
  const uint32_t id = blockIdx.x * (uint32_t)kThreads + threadIdx.x;       // below 2^32 (checked by the host)
  const uint32_t r = id / nch, c = id - r * nch;
  if (r >= rows || !selected(sel, ends, r)) return;
  const int64_t at = (int64_t)r * 2 * nch + c, aty = (int64_t)r * nch + c;
  float g[8], u[8], v[8];
  unpack8<F16>(x[at], g);
  unpack8<F16>(x[at + nch], u);
  if constexpr (BWD) {
    float d[8], dg[8], du[8];
    unpack8<F16>(dy[aty], d);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const Sig s = sigmoid(g[i]);
      const float swish = g[i] * s.s;
      v[i] = u[i] * swish;
      du[i] = d[i] * swish;
      dg[i] = d[i] * u[i] * s.s * __builtin_fmaf(g[i], s.not_s, 1.0f);
    }
    dx[at] = pack8<F16>(dg);
    dx[at + nch] = pack8<F16>(du);
    if (y != nullptr) y[aty] = pack8<F16>(v);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = u[i] * (g[i] * sigmoid(g[i]).s);
    y[aty] = pack8<F16>(v);
  }
}

template <bool BWD>
hipError_t launch(hipStream_t s, const uint16_t* dy, const uint16_t* x, int64_t rows, int64_t h,
                  const RowSelection& sel, uint16_t* dx, uint16_t* y, bool f16) {
  const dim3 grid((unsigned)((rows * (h / 8) + kThreads - 1) / kThreads)), block(kThreads);
  auto v = [](const uint16_t* p) { return reinterpret_cast<const u32x4*>(p); };
  auto w = [](uint16_t* p) { return reinterpret_cast<u32x4*>(p); };
  if (f16)
    hipLaunchKernelGGL((swiglu_kernel<true, BWD>), grid, block, 0, s, v(dy), v(x), (uint32_t)rows, (uint32_t)(h / 8),
                       sel, w(dx), w(y));
  else
    hipLaunchKernelGGL((swiglu_kernel<false, BWD>), grid, block, 0, s, v(dy), v(x), (uint32_t)rows, (uint32_t)(h / 8),
                       sel, w(dx), w(y));
  return hipGetLastError();
}

}  // namespace

hipError_t launch_swiglu(hipStream_t s, const uint16_t* x, int64_t rows, int64_t h, RowSelection sel, uint16_t* y,
                         bool f16) {
  return launch<false>(s, nullptr, x, rows, h, sel, nullptr, y, f16);
}
hipError_t launch_swiglu_backward(hipStream_t s, const uint16_t* dy, const uint16_t* x, int64_t rows, int64_t h,
                                  RowSelection sel, uint16_t* dx, uint16_t* y, bool f16) {
  return launch<true>(s, dy, x, rows, h, sel, dx, y, f16);
}

}  // namespace hq
