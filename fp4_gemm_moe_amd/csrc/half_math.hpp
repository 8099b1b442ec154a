// Matrix products of BF16 and FP16 fragments, and FP32 values as sums of 16-bit ones.
#pragma once

#include "block_gemm.hpp"

namespace hq {

typedef __bf16 v8b __attribute__((ext_vector_type(8)));
typedef short v4s __attribute__((ext_vector_type(4)));

// 16 x 16 x 32 products: lane (x, q) = (l % 16, l / 16) supplies K values 8 q ..
// + 7 of row x of w and of x, and gets rows 4 q .. + 3 (of w), column x (of x).
template <bool F16>
__device__ __forceinline__ v4f product16(v4i w, v4i x, v4f c) {
  if constexpr (F16)
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(v8h, w), __builtin_bit_cast(v8h, x), c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(v8b, w), __builtin_bit_cast(v8b, x), c, 0, 0, 0);
}

// Four rows of K at each of a 16-lane group's addresses -> four K values of the
// lane's column (the group's lane x points at columns 4 (x % 4) .. + 3 of row x / 4).
__device__ __forceinline__ v4s read_transposed(const void* lds) {
  typedef __attribute__((address_space(3))) v4s lds4;
  return __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4*)(uintptr_t)(uint32_t)(uintptr_t)(
      __attribute__((address_space(3))) const void*)lds);
}
__device__ __forceinline__ v4i join(v4s lo, v4s hi) {
  typedef short v8s __attribute__((ext_vector_type(8)));
  return __builtin_bit_cast(v4i, (v8s)__builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
}

// The top 16 bits of an FP32 value, a BF16 that is not larger; what they leave
// is exact, and zero for an infinity.
__device__ __forceinline__ float bf16_cut(float v) { return __uint_as_float(__float_as_uint(v) & 0xffff0000u); }
__device__ __forceinline__ float bf16_rest(float v, float cut) { return __builtin_fabsf(cut) == INFINITY ? 0.0f : v - cut; }

}  // namespace hq
