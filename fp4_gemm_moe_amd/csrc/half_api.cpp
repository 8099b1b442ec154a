// C-ABI layer of the 16-bit products by expert, SwiGLU in 16 bits and the
// low-rank adapters: argument validation (host only, before any device work)
// and dispatch to the kernel launchers, with the error convention of hq_api.cpp.
#include <hip/hip_runtime.h>

#include "api_util.hpp"
#include "half_internal.hpp"
#include "hq.h"

using hq::api::aligned16;
using hq::api::aligned4;
using hq::api::current_device;
using hq::api::fail;
using hq::api::kI32;
using hq::api::launched;
using hq::api::ok;

namespace {

constexpr int64_t kMaxPlaces = (int64_t)1 << 30;     // places and tokens of an adapters' batch
constexpr int64_t kMaxWidth = (int64_t)1 << 21;      // 256 rows of it stay below 2^31 bytes

hq_status check_groups(const char* what, int32_t num_groups) {
  if (num_groups < 1 || num_groups > 1024)
    return fail(HQ_ERR_SHAPE, "%s: %d groups: must be in [1, 1024]", what, num_groups);
  return HQ_OK;
}

// A width of 16-bit rows: whole 16-byte words.
hq_status check_width(const char* what, const char* name, int64_t w, int64_t least) {
  if (w < least || w % 8 != 0 || w >= kMaxWidth)
    return fail(HQ_ERR_SHAPE, "%s: %s=%lld must be a multiple of 8 in [%lld, 2^21)", what, name, (long long)w,
                (long long)least);
  return HQ_OK;
}

// Checks common to the products; p holds the shape.  reads: a and b are read.
hq_status check_product(const char* what, uint32_t flags, uint32_t allowed, hq::HalfGemmArgs& p, bool reads,
                        bool* noop) {
  *noop = false;
  if ((flags & ~allowed) != 0) return fail(HQ_ERR_MODE, "%s: unknown flags 0x%x", what, flags);
  if ((flags & HQ_ACCUMULATE) && !(flags & HQ_OUT_FP32))
    return fail(HQ_ERR_MODE, "%s: HQ_ACCUMULATE needs HQ_OUT_FP32", what);
  p.f16 = (flags & HQ_IN_FP16) != 0;
  p.b_t = (flags & HQ_TRANSPOSE) != 0;
  p.out_kind = (flags & HQ_ACCUMULATE) ? hq::kOutF32Add
               : (flags & HQ_OUT_FP32) ? hq::kOutF32
               : p.f16                 ? hq::kOutF16
                                       : hq::kOutBf16;
  if (p.rows < 0 || p.rows > kI32) return fail(HQ_ERR_SHAPE, "%s: row counts must be in [0, 2^31)", what);
  if ((p.rows / 16 + p.groups + 1) * (p.n / 16 + 1) * (p.form == hq::kGroupK ? p.groups : 1) > kI32)
    return fail(HQ_ERR_SHAPE, "%s: problem too large (tile count exceeds 2^31)", what);
  if (p.rows == 0 || p.n == 0) {
    *noop = true;
    return HQ_OK;
  }
  if (!p.out || (reads && (!p.a || !p.b))) return fail(HQ_ERR_NULL, "%s: a, b and out are required", what);
  if (!aligned16(p.a) || !aligned16(p.b) || !aligned16(p.out))
    return fail(HQ_ERR_ALIGN, "%s: a, b and out must be 16-byte aligned", what);
  return HQ_OK;
}

hq_status run_product(const char* what, void* stream, const hq::HalfGemmArgs& p) {
  hq::DeviceInfo dev;
  const hq_status st = current_device(&dev);
  if (st != HQ_OK) return st;
  return launched(hq::launch_half_gemm((hipStream_t)stream, p, dev), what);
}

hq_status check_selection(const char* what, int64_t rows, int64_t h, const hq::RowSelection& sel) {
  if (h <= 0 || h % 8 != 0 || h > kI32 / 16)
    return fail(HQ_ERR_SHAPE, "%s: h=%lld must be a positive multiple of 8 below 2^27", what, (long long)h);
  if (rows < 0 || rows > kI32) return fail(HQ_ERR_SHAPE, "%s: rows=%lld out of range", what, (long long)rows);
  if (rows > 0 && h / 8 > (hq::kMaxWorkItems - 256) / rows)
    return fail(HQ_ERR_SHAPE, "%s: problem too large: rows * h must be below 2^35", what);
  if (sel.groups == 0) {
    if (sel.group_end != nullptr || sel.valid != nullptr)
      return fail(HQ_ERR_SHAPE, "%s: group_end and valid need num_groups", what);
    return HQ_OK;
  }
  const hq_status st = check_groups(what, sel.groups);
  if (st != HQ_OK) return st;
  if (sel.group_end == nullptr && sel.slot_rows <= 0)
    return fail(HQ_ERR_SHAPE, "%s: slot_rows must be > 0 when group_end is NULL", what);
  if (!aligned4(sel.group_end) || !aligned4(sel.valid))
    return fail(HQ_ERR_ALIGN, "%s: group_end and valid must be 4-byte aligned", what);
  return HQ_OK;
}

hq_status check_lora_shape(const char* what, int64_t max_rows, int64_t n, int64_t k, int64_t r, int32_t adapters) {
  hq_status st = check_groups(what, adapters);
  if (st != HQ_OK) return st;
  if ((st = check_width(what, "n", n, 8)) != HQ_OK) return st;
  if ((st = check_width(what, "k", k, 8)) != HQ_OK) return st;
  if (r < 8 || r % 8 != 0 || r > 512)
    return fail(HQ_ERR_SHAPE, "%s: r=%lld must be a multiple of 8 in [8, 512]", what, (long long)r);
  if (max_rows < 0 || max_rows >= kMaxPlaces)
    return fail(HQ_ERR_SHAPE, "%s: max_rows=%lld must be in [0, 2^30)", what, (long long)max_rows);
  return HQ_OK;
}

// Checks common to both directions, after the shape's.
hq_status check_lora(const char* what, const hq::LoraArgs& p, bool backward, uint64_t need, uint64_t workspace_bytes) {
  const hq::LoraPlan& pl = p.plan;
  if (pl.m < 0 || pl.m >= kMaxPlaces) return fail(HQ_ERR_SHAPE, "%s: m=%lld must be in [0, 2^30)", what, (long long)pl.m);
  if (hq::lora_work_items(p, backward) >= hq::kMaxWorkItems)
    return fail(HQ_ERR_SHAPE, "%s: problem too large (a launch would pass 2^32 work items)", what);
  if ((pl.row_map != nullptr) != (pl.row_pair != nullptr) && pl.m > 0 && pl.max_rows > 0)
    return fail(HQ_ERR_NULL, "%s: row_map and row_pair go together", what);
  const bool no_places = pl.row_map != nullptr && pl.max_rows == 0;      // row_pair is empty, and may be NULL
  if (pl.row_pair == nullptr && pl.max_rows != pl.m && !no_places)
    return fail(HQ_ERR_SHAPE, "%s: without row_pair max_rows=%lld must be m=%lld", what, (long long)pl.max_rows,
                (long long)pl.m);
  if (!pl.group_end) return fail(HQ_ERR_NULL, "%s: group_end is required", what);
  if (need > 0 && p.workspace == nullptr) return fail(HQ_ERR_NULL, "%s: this shape needs a workspace", what);
  if (workspace_bytes < need)
    return fail(HQ_ERR_SHAPE, "%s: workspace_bytes=%llu, this shape needs %llu", what,
                (unsigned long long)workspace_bytes, (unsigned long long)need);
  if (!aligned16(p.x) || !aligned16(p.dy) || !aligned16(p.a) || !aligned16(p.b) || !aligned16(p.base) ||
      !aligned16(p.out) || !aligned16(p.v) || !aligned16(p.da) || !aligned16(p.db) || !aligned16(p.workspace))
    return fail(HQ_ERR_ALIGN, "%s: 16-bit tensors, v, da, db and the workspace must be 16-byte aligned", what);
  if (!aligned4(pl.row_map) || !aligned4(pl.row_pair) || !aligned4(pl.group_end) || !aligned4(pl.scale))
    return fail(HQ_ERR_ALIGN, "%s: row_map, row_pair, group_end and scale must be 4-byte aligned", what);
  return HQ_OK;
}

}  // namespace

extern "C" {

hq_status hq_half_group_contiguous_gemm(void* stream, uint32_t flags, const uint16_t* a, const uint16_t* b,
                                        const int32_t* group_end, int32_t num_groups, void* out, int64_t m_total,
                                        int64_t n, int64_t k) {
  const char* what = "hq_half_group_contiguous_gemm";
  hq_status st = check_groups(what, num_groups);
  if (st != HQ_OK) return st;
  if ((st = check_width(what, "n", n, 0)) != HQ_OK) return st;
  if ((st = check_width(what, "k", k, 8)) != HQ_OK) return st;
  hq::HalfGemmArgs p{a, b, out, group_end, nullptr, m_total, 0, n, k, num_groups, hq::kContiguous};
  bool noop;
  if ((st = check_product(what, flags, HQ_IN_FP16 | HQ_TRANSPOSE | HQ_OUT_FP32 | HQ_ACCUMULATE, p, true, &noop)) !=
      HQ_OK)
    return st;
  if (noop) return ok();
  if (!group_end) return fail(HQ_ERR_NULL, "%s: group_end is required", what);
  if (!aligned4(group_end)) return fail(HQ_ERR_ALIGN, "%s: group_end must be 4-byte aligned", what);
  return run_product(what, stream, p);
}

hq_status hq_half_group_masked_gemm(void* stream, uint32_t flags, const uint16_t* a, const uint16_t* b,
                                    const int32_t* masked_m, int32_t num_groups, int64_t max_m_per_group, void* out,
                                    int64_t n, int64_t k) {
  const char* what = "hq_half_group_masked_gemm";
  hq_status st = check_groups(what, num_groups);
  if (st != HQ_OK) return st;
  if (max_m_per_group <= 0 || max_m_per_group > kI32 / num_groups)
    return fail(HQ_ERR_SHAPE, "%s: max_m_per_group=%lld must be > 0 and num_groups * max_m below 2^31", what,
                (long long)max_m_per_group);
  if ((st = check_width(what, "n", n, 0)) != HQ_OK) return st;
  if ((st = check_width(what, "k", k, 8)) != HQ_OK) return st;
  hq::HalfGemmArgs p{a, b, out, nullptr, masked_m, num_groups * max_m_per_group, max_m_per_group, n, k, num_groups,
                     hq::kMasked};
  bool noop;
  if ((st = check_product(what, flags, HQ_IN_FP16 | HQ_TRANSPOSE | HQ_OUT_FP32 | HQ_ACCUMULATE, p, true, &noop)) !=
      HQ_OK)
    return st;
  if (noop) return ok();
  if (!masked_m) return fail(HQ_ERR_NULL, "%s: masked_m is required", what);
  if (!aligned4(masked_m)) return fail(HQ_ERR_ALIGN, "%s: masked_m must be 4-byte aligned", what);
  return run_product(what, stream, p);
}

hq_status hq_half_group_k_gemm(void* stream, uint32_t flags, const uint16_t* a, const uint16_t* b,
                               const int32_t* group_end, int32_t num_groups, void* out, int64_t m, int64_t n,
                               int64_t rows) {
  const char* what = "hq_half_group_k_gemm";
  hq_status st = check_groups(what, num_groups);
  if (st != HQ_OK) return st;
  if ((st = check_width(what, "m", m, 0)) != HQ_OK) return st;
  if ((st = check_width(what, "n", n, 0)) != HQ_OK) return st;
  if (rows < 0 || rows > kI32) return fail(HQ_ERR_SHAPE, "%s: rows=%lld must be in [0, 2^31)", what, (long long)rows);
  hq::HalfGemmArgs p{a, b, out, group_end, nullptr, m, 0, n, rows, num_groups, hq::kGroupK};
  bool noop;
  if ((st = check_product(what, flags, HQ_IN_FP16 | HQ_OUT_FP32 | HQ_ACCUMULATE, p, rows > 0, &noop)) != HQ_OK)
    return st;
  if (noop) return ok();
  if (!group_end) return fail(HQ_ERR_NULL, "%s: group_end is required", what);
  if (!aligned4(group_end)) return fail(HQ_ERR_ALIGN, "%s: group_end must be 4-byte aligned", what);
  return run_product(what, stream, p);
}

hq_status hq_swiglu(void* stream, const uint16_t* x, int64_t rows, int64_t h, int32_t num_groups,
                    const int32_t* group_end, int64_t slot_rows, const int32_t* valid, uint16_t* y, uint32_t flags) {
  const char* what = "hq_swiglu";
  if ((flags & ~HQ_IN_FP16) != 0) return fail(HQ_ERR_MODE, "%s: unknown flags 0x%x", what, flags);
  const hq::RowSelection sel{num_groups, group_end, slot_rows, valid};
  hq_status st = check_selection(what, rows, h, sel);
  if (st != HQ_OK) return st;
  if (rows == 0) return ok();
  if (!x || !y) return fail(HQ_ERR_NULL, "%s: x and y are required", what);
  if (!aligned16(x) || !aligned16(y)) return fail(HQ_ERR_ALIGN, "%s: x and y must be 16-byte aligned", what);
  hq::DeviceInfo dev;
  if ((st = current_device(&dev)) != HQ_OK) return st;
  return launched(hq::launch_swiglu((hipStream_t)stream, x, rows, h, sel, y, (flags & HQ_IN_FP16) != 0), what);
}

hq_status hq_swiglu_backward(void* stream, const uint16_t* dy, const uint16_t* x, int64_t rows, int64_t h,
                             int32_t num_groups, const int32_t* group_end, int64_t slot_rows, const int32_t* valid,
                             uint16_t* dx, uint16_t* y, uint32_t flags) {
  const char* what = "hq_swiglu_backward";
  if ((flags & ~HQ_IN_FP16) != 0) return fail(HQ_ERR_MODE, "%s: unknown flags 0x%x", what, flags);
  const hq::RowSelection sel{num_groups, group_end, slot_rows, valid};
  hq_status st = check_selection(what, rows, h, sel);
  if (st != HQ_OK) return st;
  if (rows == 0) return ok();
  if (!dy || !x || !dx) return fail(HQ_ERR_NULL, "%s: dy, x and dx are required", what);
  if (!aligned16(dy) || !aligned16(x) || !aligned16(dx) || !aligned16(y))
    return fail(HQ_ERR_ALIGN, "%s: dy, x, dx and y must be 16-byte aligned", what);
  hq::DeviceInfo dev;
  if ((st = current_device(&dev)) != HQ_OK) return st;
  return launched(hq::launch_swiglu_backward((hipStream_t)stream, dy, x, rows, h, sel, dx, y,
                                             (flags & HQ_IN_FP16) != 0),
                  what);
}

hq_status hq_lora_workspace_size(int64_t max_rows, int64_t n, int64_t k, int64_t r, int32_t num_adapters,
                                 uint64_t* bytes) {
  const char* what = "hq_lora_workspace_size";
  if (bytes == nullptr) return fail(HQ_ERR_NULL, "%s: bytes is required", what);
  const hq_status st = check_lora_shape(what, max_rows, n, k, r, num_adapters);
  if (st != HQ_OK) return st;
  *bytes = hq::lora_workspace_bytes(max_rows, n, k, r, num_adapters);
  return ok();
}

hq_status hq_lora(void* stream, uint32_t flags, const uint16_t* x, const uint16_t* a, const uint16_t* b,
                  const float* scale, const int32_t* group_end, int32_t num_adapters, const int32_t* row_map,
                  const int32_t* row_pair, int64_t max_rows, const uint16_t* base, uint16_t* out, float* v, int64_t m,
                  int64_t n, int64_t k, int64_t r, void* workspace, uint64_t workspace_bytes) {
  const char* what = "hq_lora";
  if ((flags & ~HQ_IN_FP16) != 0) return fail(HQ_ERR_MODE, "%s: unknown flags 0x%x", what, flags);
  hq_status st = check_lora_shape(what, max_rows, n, k, r, num_adapters);
  if (st != HQ_OK) return st;
  hq::LoraArgs p{};
  p.plan = hq::LoraPlan{group_end, row_map, row_pair, scale, max_rows, m, num_adapters};
  p.x = x;
  p.a = a;
  p.b = b;
  p.base = base;
  p.out = out;
  p.v = v;
  p.n = n;
  p.k = k;
  p.r = r;
  p.f16 = (flags & HQ_IN_FP16) != 0;
  p.workspace = workspace;
  if ((st = check_lora(what, p, false, hq::lora_workspace_bytes(max_rows, n, k, r, num_adapters), workspace_bytes)) !=
      HQ_OK)
    return st;
  if (m == 0) return ok();
  if (!x || !a || !b || !out) return fail(HQ_ERR_NULL, "%s: x, a, b and out are required", what);
  hq::DeviceInfo dev;
  if ((st = current_device(&dev)) != HQ_OK) return st;
  return launched(hq::launch_lora((hipStream_t)stream, p), what);
}

hq_status hq_lora_backward_workspace_size(int64_t max_rows, int64_t n, int64_t k, int64_t r, int32_t num_adapters,
                                          uint64_t* bytes) {
  const char* what = "hq_lora_backward_workspace_size";
  if (bytes == nullptr) return fail(HQ_ERR_NULL, "%s: bytes is required", what);
  const hq_status st = check_lora_shape(what, max_rows, n, k, r, num_adapters);
  if (st != HQ_OK) return st;
  *bytes = hq::lora_backward_workspace_bytes(max_rows, n, k, r, num_adapters);
  return ok();
}

hq_status hq_lora_backward(void* stream, uint32_t flags, const uint16_t* dy, const uint16_t* x, const float* v,
                           const uint16_t* a, const uint16_t* b, const float* scale, const int32_t* group_end,
                           int32_t num_adapters, const int32_t* row_map, const int32_t* row_pair, int64_t max_rows,
                           const uint16_t* base, uint16_t* dx, float* da, float* db, int64_t m, int64_t n, int64_t k,
                           int64_t r, void* workspace, uint64_t workspace_bytes) {
  const char* what = "hq_lora_backward";
  if ((flags & ~(HQ_IN_FP16 | HQ_ACCUMULATE)) != 0) return fail(HQ_ERR_MODE, "%s: unknown flags 0x%x", what, flags);
  hq_status st = check_lora_shape(what, max_rows, n, k, r, num_adapters);
  if (st != HQ_OK) return st;
  hq::LoraArgs p{};
  p.plan = hq::LoraPlan{group_end, row_map, row_pair, scale, max_rows, m, num_adapters};
  p.x = x;
  p.a = a;
  p.b = b;
  p.base = base;
  p.out = dx;
  p.v = const_cast<float*>(v);
  p.n = n;
  p.k = k;
  p.r = r;
  p.f16 = (flags & HQ_IN_FP16) != 0;
  p.dy = dy;
  p.da = da;
  p.db = db;
  p.accumulate = (flags & HQ_ACCUMULATE) != 0;
  p.workspace = workspace;
  if ((st = check_lora(what, p, true, hq::lora_backward_workspace_bytes(max_rows, n, k, r, num_adapters),
                       workspace_bytes)) != HQ_OK)
    return st;
  if (base != nullptr && dx == nullptr) return fail(HQ_ERR_NULL, "%s: base needs dx", what);
  if (!da || !db || (m > 0 && (!dy || !x || !a || !b)) || (m > 0 && max_rows > 0 && !v))
    return fail(HQ_ERR_NULL, "%s: dy, x, v, a, b, da and db are required", what);
  if (m == 0) p.plan.max_rows = 0;          // no place holds a token: the sums are empty
  hq::DeviceInfo dev;
  if ((st = current_device(&dev)) != HQ_OK) return st;
  return launched(hq::launch_lora_backward((hipStream_t)stream, p), what);
}

}  // extern "C"
