// Block-128 FP8: the scale and code rule shared by the kernels that write
// block-quantised values.
//
// A block (1 x 128 of a row, or 128 x 128) of values x has one FP32 scale
//   s = max(amax / 448, 2^-126)            (IEEE FP32 division)
// and E4M3 codes of x / s (IEEE FP32 quotient, nearest even, saturating at
// 448; the sign is kept, also for zero).  448 is E4M3's largest value, so the
// block's largest magnitude uses the whole range.  The floor 2^-126 keeps s
// normal for zero and near-zero blocks.  A block that holds an infinity gets
// s = Inf, codes 0 for its finite values and NaN for the infinities; a block
// that holds a NaN gets s = NaN and NaN codes: either way its products are
// NaN, not silently finite.
#pragma once

#include "fmt.hpp"

namespace hq {

// 16-byte store, with the non-temporal policy if NT.  Outputs of more than
// kStreamBytes, which the 256 MB Infinity Cache would not keep for their
// reader, are stored so: [65536, 4096] codes 137 -> 133 us, the combination's
// gradient of 4096 tokens top 8 of 4096 120 -> 112 us; smaller ones are not
// ([16384, 4096] codes 33.8 us, 34.8 us non-temporal).
constexpr int64_t kStreamBytes = (int64_t)128 << 20;
template <bool NT>
__device__ __forceinline__ void store16(void* p, const u32x4& v) {
  if constexpr (NT) __builtin_nontemporal_store(v, static_cast<u32x4*>(p));
  else *static_cast<u32x4*>(p) = v;
}

// FP16 halves of a packed dword -> FP32 (exact).
__device__ __forceinline__ float f16_lo(uint32_t w) { return (float)__builtin_bit_cast(_Float16, (uint16_t)w); }
__device__ __forceinline__ float f16_hi(uint32_t w) {
  return (float)__builtin_bit_cast(_Float16, (uint16_t)(w >> 16));
}

// Two values of a packed dword of BF16 or FP16.
template <bool F16>
__device__ __forceinline__ float half_lo(uint32_t w) {
  if constexpr (F16) return f16_lo(w);
  else return bf16_lo(w);
}
template <bool F16>
__device__ __forceinline__ float half_hi(uint32_t w) {
  if constexpr (F16) return f16_hi(w);
  else return bf16_hi(w);
}

// Two FP32 values -> a packed dword of BF16 or FP16, nearest even.
template <bool F16>
__device__ __forceinline__ uint32_t pack_half2(float a, float b) {
  typedef float f32x2 __attribute__((ext_vector_type(2)));
  if constexpr (F16) {
    typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
    return __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2{a, b}), f16x2));
  } else {
    typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
    return __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2{a, b}), bf16x2));
  }
}

// The block scale from the FP32 pattern of the block's largest magnitude
// (integer order equals float order for non-negative patterns, with Inf above
// every finite value and NaN above Inf).
__device__ __forceinline__ float block_scale(uint32_t amax_bits) {
  const float s = __uint_as_float(amax_bits) / 448.0f;
  return s < 0x1p-126f ? 0x1p-126f : s;      // false for NaN: a NaN stays
}

// N (a multiple of 4) values -> E4M3 codes of x / s, four to a dword.  For s
// in [2^-56, 2^56] the quotients share one reciprocal: r = rcp(s) with a
// Newton step, then t = x r and two FMA residual corrections
// t -= (s t - x) r, which give the correctly rounded quotient (P. Markstein,
// "IA-64 and Elementary Functions", 2000) wherever it can round to anything
// but a zero code; with the residual's sign this way round, a zero keeps x's
// sign.  These quotients are at most 448 (1 + 2^-23), which rounds to 448, so
// only other scales, which take the IEEE division, clamp theirs.
template <int N>
__device__ __forceinline__ void block_codes(const float (&x)[N], float s, uint32_t (&w)[N / 4]) {
  float q[N];
  if (s >= 0x1p-56f && s <= 0x1p56f) {
    float r = __builtin_amdgcn_rcpf(s);
    r = __builtin_fmaf(__builtin_fmaf(-s, r, 1.0f), r, r);
#pragma unroll
    for (int i = 0; i < N; ++i) {
      float t = x[i] * r;
      t = __builtin_fmaf(__builtin_fmaf(s, t, -x[i]), -r, t);
      q[i] = __builtin_fmaf(__builtin_fmaf(s, t, -x[i]), -r, t);
    }
  } else if (s <= 0x1p127f) {
#pragma unroll
    for (int i = 0; i < N; ++i) q[i] = __builtin_amdgcn_fmed3f(x[i] / s, -448.0f, 448.0f);
  } else {                                     // s is Inf or NaN
#pragma unroll
    for (int i = 0; i < N; ++i) q[i] = x[i] / s;
  }
#pragma unroll
  for (int i = 0; i < N / 4; ++i) {
    const int v = __builtin_amdgcn_cvt_pk_fp8_f32(q[4 * i], q[4 * i + 1], 0, false);
    w[i] = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(q[4 * i + 2], q[4 * i + 3], v, true);
  }
}

// Largest magnitudes of packed BF16 or FP16 pairs, as a packed pair: the
// patterns without their signs, in integer order (NaN above Inf above the rest).
__device__ __forceinline__ uint32_t abs_max2(uint32_t m, uint32_t w) {
  typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));
  return __builtin_bit_cast(uint32_t, __builtin_elementwise_max(__builtin_bit_cast(u16x2, m),
                                                                __builtin_bit_cast(u16x2, w & 0x7fff7fffu)));
}

// The FP32 pattern of the larger half of such a pair.
template <bool F16>
__device__ __forceinline__ uint32_t abs_max_bits(uint32_t m) {
  const uint32_t h = (m & 0xffffu) > m >> 16 ? m & 0xffffu : m >> 16;
  return __float_as_uint(half_lo<F16>(h));
}

// Largest |x| pattern of 16 packed values.
template <bool F16>
__device__ __forceinline__ uint32_t abs_max(const uint4& u, const uint4& v) {
  uint32_t m = abs_max2(u.x & 0x7fff7fffu, u.y);
  m = abs_max2(abs_max2(m, u.z), u.w);
  m = abs_max2(abs_max2(m, v.x), v.y);
  return abs_max_bits<F16>(abs_max2(abs_max2(m, v.z), v.w));
}

// Largest |x| pattern of N values.
template <int N>
__device__ __forceinline__ uint32_t abs_max(const float (&x)[N]) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const uint32_t a = __float_as_uint(x[i]) & 0x7fffffffu;
    m = a > m ? a : m;
  }
  return m;
}

// Max over the 8 lanes of an aligned lane octet.
__device__ __forceinline__ uint32_t octet_max_u32(uint32_t v) {
  v = quad_max_u32(v);
  const uint32_t t = (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x141, 0xF, 0xF, false);   // row_half_mirror
  return v > t ? v : t;
}

// Sixteen values from two 16-byte words of packed BF16 or FP16.
template <bool F16>
__device__ __forceinline__ void unpack16(const uint4& u, const uint4& v, float (&f)[16]) {
  const uint32_t w[8] = {u.x, u.y, u.z, u.w, v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    f[2 * i] = half_lo<F16>(w[i]);
    f[2 * i + 1] = half_hi<F16>(w[i]);
  }
}

}  // namespace hq
