// Internal interfaces of the 16-bit products by expert, SwiGLU in 16 bits and
// the low-rank adapters: what their C-ABI layer (half_api.cpp) passes to the
// kernel translation units.  Nothing here is exported.
#pragma once

#include "block_internal.hpp"

namespace hq {

// out[r] = a[r] b[g]^T (or a[r] b[g]) over GroupForm's kContiguous or kMasked
// rows, or, for kGroupK, out[g] = sum over the rows of g of a[r]^T b[r].
struct HalfGemmArgs {
  const uint16_t* a;         // [rows, k] (kGroupK: [k, rows])
  const uint16_t* b;         // [groups, n, k]; b_t: [groups, k, n] (kGroupK: [k, n])
  void* out;                 // [rows, n] (kGroupK: [groups, rows, n])
  const int32_t* group_end;  // kContiguous: row ends; kGroupK: ends along k
  const int32_t* counts;     // kMasked
  int64_t rows;
  int64_t slot_rows;         // kMasked
  int64_t n, k;
  int32_t groups;
  int32_t form;
  int32_t out_kind;          // BlockOut
  bool b_t, f16;
  bool stream;               // tiled kernel: results leave past the caches
};
hipError_t launch_half_gemm(hipStream_t s, const HalfGemmArgs& args, const DeviceInfo& dev);

// Rows that a SwiGLU call takes: all of them (groups == 0), or by group.
struct RowSelection {
  int32_t groups;
  const int32_t* group_end;  // nullptr: slots of slot_rows
  int64_t slot_rows;
  const int32_t* valid;      // nullptr: all rows of a group
};
hipError_t launch_swiglu(hipStream_t s, const uint16_t* x, int64_t rows, int64_t h, RowSelection sel, uint16_t* y,
                         bool f16);
hipError_t launch_swiglu_backward(hipStream_t s, const uint16_t* dy, const uint16_t* x, int64_t rows, int64_t h,
                                  RowSelection sel, uint16_t* dx, uint16_t* y, bool f16);

// Tokens by adapter: place i of adapter g, in [group_end[g - 1], group_end[g]),
// holds token row_pair[i] (i itself where row_pair is nullptr).
struct LoraPlan {
  const int32_t* group_end;
  const int32_t* row_map;
  const int32_t* row_pair;
  const float* scale;        // nullptr: 1
  int64_t max_rows;
  int64_t m;
  int32_t adapters;
};
struct LoraArgs {
  LoraPlan plan;
  const uint16_t *x, *a, *b, *base;
  uint16_t* out;             // backward: dx
  float* v;                  // backward: read
  int64_t n, k, r;
  bool f16;
  // backward
  const uint16_t* dy;
  float *da, *db;
  bool accumulate;
  void* workspace;
};
int64_t lora_work_items(const LoraArgs& args, bool backward);
uint64_t lora_workspace_bytes(int64_t max_rows, int64_t n, int64_t k, int64_t r, int32_t adapters);
uint64_t lora_backward_workspace_bytes(int64_t max_rows, int64_t n, int64_t k, int64_t r, int32_t adapters);
hipError_t launch_lora(hipStream_t s, const LoraArgs& args);
hipError_t launch_lora_backward(hipStream_t s, const LoraArgs& args);

}  // namespace hq
