// Internal interfaces of the block-128 FP8 products and the token dispatch:
// what their C-ABI layer (block_api.cpp) passes to the kernel translation
// units.  Nothing here is exported.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "hq_internal.hpp"

namespace hq {

enum BlockOut : int32_t { kOutBf16 = 0, kOutF16 = 1, kOutF32 = 2, kOutF32Add = 3 };
// GroupForm's forms, and the product that sums over the groups' K ranges.
constexpr int32_t kGroupK = 3;

// Which accesses of a tiled launch take the non-temporal policy: none, the
// stores of results, or those and the loads of b.
enum BlockPolicy : int32_t { kPolKeep = 0, kPolStreamOut = 1, kPolStreamAll = 2 };

// out[r, n] = sum over K blocks of sa[r, kb] sb[n / 128, kb] (a[r] . b[n])_kb,
// in one of the forms of GroupForm or kGroupK.
struct BlockGemmArgs {
  const uint8_t* a;          // [rows, k] E4M3
  const float* sa;           // [rows, nkb]
  const uint8_t* b;          // [groups, n, k] E4M3 (kGroupK: [n, k])
  const float* sb;           // [groups, nnb, nkb] (kGroupK: [nnb, nkb])
  void* out;                 // [rows, n] (kGroupK: [groups, rows, n])
  const int32_t* group_end;  // kContiguous: row ends; kGroupK: ends along k
  const int32_t* counts;     // kMasked
  int64_t rows;              // rows of a (all groups)
  int64_t slot_rows;         // kUniform, kMasked: rows of a group
  int64_t n, k;
  int64_t ldo;               // elements from row to row of out
  int32_t nkb, nnb;          // ceil(k / 128), ceil(n / 128)
  int32_t groups;
  int32_t form;
  int32_t out_kind;          // BlockOut
  int32_t slices;            // kUniform: K slices; out then holds [slices, rows, n] FP32 partial sums
};

// A launch holds fewer than 2^32 work items along a dimension of its grid.  The
// functions below say how many workgroups a call takes; the C-ABI layer refuses
// calls that do not fit, so the kernels' workgroup numbers are below 2^24 (256
// threads a workgroup) and 128-blocks of a row form below 2^29.
constexpr int64_t kMaxWorkItems = (int64_t)1 << 32;

// 256 threads: 32 blocks of 1 x 128, or one 128 x 128 tile.
constexpr int kQuantThreads = 256;
inline int64_t quant_row_groups(int64_t rows, int64_t k) { return (rows * ((k + 127) / 128) + 31) / 32; }
inline int64_t quant_tile_groups(int64_t batch, int64_t m, int64_t k) {
  return batch * ((m + 127) / 128) * ((k + 127) / 128);
}

hipError_t launch_block_gemm(hipStream_t s, const BlockGemmArgs& args, const DeviceInfo& dev, void* workspace,
                             uint64_t workspace_bytes);
// Bytes of workspace that a dense or batch call of this shape uses.
uint64_t block_gemm_workspace_bytes(const BlockGemmArgs& args, const DeviceInfo& dev);

hipError_t launch_block_quant(hipStream_t s, const uint16_t* x, int64_t batch, int64_t m, int64_t k, uint8_t* q,
                              float* sf, bool two_d, bool transpose, bool fp16);
hipError_t launch_swiglu_block_quant(hipStream_t s, const uint16_t* x, int64_t rows, int64_t h,
                                     const int32_t* last_end, uint8_t* q, float* sf, bool fp16);

uint64_t moe_sort_workspace_bytes(int64_t pairs, int32_t experts);
hipError_t launch_moe_sort(hipStream_t s, const int64_t* ids, int64_t pairs, int32_t experts, int32_t align,
                           int64_t max_rows, int32_t* row_map, int32_t* row_pair, int32_t* group_end,
                           int32_t* counts, void* workspace);
// The rows of groups past their counts (padding): where they lie, and how
// many there are, on the device.
struct PadRows {
  const int32_t* group_end;   // nullptr: no padding rows are written
  const int32_t* counts;
  int32_t groups;
};
// Four units of 64 lanes a workgroup of 256 threads: pieces of `piece` bytes or
// values of every token's row; then kPadParts workgroups for each group's
// padding rows.
constexpr int kMoeThreads = 256;
constexpr int kPadParts = 8;
inline int64_t pad_groups(const PadRows& pad) { return pad.group_end != nullptr ? (int64_t)pad.groups * kPadParts : 0; }
inline int64_t piece_groups(int64_t tokens, int64_t width, int64_t piece) {
  return (tokens * ((width + piece - 1) / piece) + 3) / 4;
}
// The combination's gradient: a workgroup a token, a wave for each of its slots
// (four waves at least, for the padding rows, and eight at most).
inline int combine_bwd_waves(int topk) { return topk > 8 ? 8 : (topk < 4 ? 4 : topk); }
hipError_t launch_moe_permute(hipStream_t s, const uint8_t* x, int64_t tokens, int64_t row_bytes,
                              const int32_t* row_map, int32_t topk, PadRows pad, int64_t max_rows, uint8_t* out);
hipError_t launch_moe_permute_block_quant(hipStream_t s, const uint16_t* x, int64_t tokens, int64_t h,
                                          const int32_t* row_map, int32_t topk, PadRows pad, int64_t max_rows,
                                          uint8_t* q, float* sf, bool fp16);
hipError_t launch_moe_combine(hipStream_t s, const uint16_t* y, int64_t tokens, int64_t h, const int32_t* row_map,
                              int32_t topk, const float* weights, int64_t max_rows, uint16_t* out, bool fp16);
hipError_t launch_moe_combine_backward(hipStream_t s, const uint16_t* dout, const uint16_t* y, int64_t tokens,
                                       int64_t h, const int32_t* row_map, int32_t topk, const float* weights,
                                       PadRows pad, int64_t max_rows, uint16_t* dy, float* dweights, bool fp16);

}  // namespace hq
