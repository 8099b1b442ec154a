// C-ABI layer of the block-128 FP8 products and the token dispatch: argument
// validation (host only, before any device work) and dispatch to the kernel
// launchers, with the error convention of hq_api.cpp.
#include <hip/hip_runtime.h>

#include "api_util.hpp"
#include "block_internal.hpp"
#include "hq.h"

using hq::api::aligned16;
using hq::api::aligned4;
using hq::api::aligned8;
using hq::api::current_device;
using hq::api::fail;
using hq::api::kI32;
using hq::api::launched;
using hq::api::ok;

namespace {

constexpr uint32_t kOutFlags = HQ_OUT_FP16 | HQ_OUT_FP32 | HQ_ACCUMULATE;

// Checks common to the products; p holds the shape, rows those of a.
hq_status check_product(const char* what, uint32_t flags, hq::BlockGemmArgs& p, bool* noop) {
  *noop = false;
  if ((flags & ~kOutFlags) != 0) return fail(HQ_ERR_MODE, "%s: unknown flags 0x%x", what, flags);
  if ((flags & HQ_OUT_FP16) && (flags & HQ_OUT_FP32))
    return fail(HQ_ERR_MODE, "%s: HQ_OUT_FP16 and HQ_OUT_FP32 exclude each other", what);
  if ((flags & HQ_ACCUMULATE) && !(flags & HQ_OUT_FP32))
    return fail(HQ_ERR_MODE, "%s: HQ_ACCUMULATE needs HQ_OUT_FP32", what);
  if (p.k <= 0 || p.k % 32 != 0)
    return fail(HQ_ERR_SHAPE, "%s: k=%lld must be a positive multiple of 32", what, (long long)p.k);
  if (p.n < 0 || p.n % 8 != 0)
    return fail(HQ_ERR_SHAPE, "%s: n=%lld must be a non-negative multiple of 8", what, (long long)p.n);
  if (p.rows < 0) return fail(HQ_ERR_SHAPE, "%s: negative row count", what);
  if (p.rows > kI32 || p.n > kI32 || p.k > kI32)
    return fail(HQ_ERR_SHAPE, "%s: dimensions must be below 2^31", what);
  // a tile's operand offsets (up to 256 rows) are 32-bit
  if (p.k > kI32 / 256) return fail(HQ_ERR_SHAPE, "%s: k=%lld: 256 * k must be below 2^31", what, (long long)p.k);
  if ((p.rows / 16 + p.groups + 1) * (p.n / 16 + 1) > kI32)
    return fail(HQ_ERR_SHAPE, "%s: problem too large (tile count exceeds 2^31)", what);
  p.nkb = (int32_t)((p.k + 127) / 128);
  p.nnb = (int32_t)((p.n + 127) / 128);
  p.out_kind = (flags & HQ_ACCUMULATE) ? hq::kOutF32Add
               : (flags & HQ_OUT_FP32) ? hq::kOutF32
               : (flags & HQ_OUT_FP16) ? hq::kOutF16
                                       : hq::kOutBf16;
  p.slices = 1;
  if (p.rows == 0 || p.n == 0) {
    *noop = true;
    return HQ_OK;
  }
  if (!p.a || !p.sa || !p.b || !p.sb || !p.out)
    return fail(HQ_ERR_NULL, "%s: a, sfa, b, sfb and out are required", what);
  if (!aligned16(p.a) || !aligned16(p.b) || !aligned16(p.out))
    return fail(HQ_ERR_ALIGN, "%s: a, b and out must be 16-byte aligned", what);
  if (!aligned4(p.sa) || !aligned4(p.sb)) return fail(HQ_ERR_ALIGN, "%s: sfa and sfb must be 4-byte aligned", what);
  return HQ_OK;
}

hq::BlockGemmArgs product(const uint8_t* a, const float* sfa, const uint8_t* b, const float* sfb, void* out,
                          int64_t rows, int64_t n, int64_t k, int32_t groups, int32_t form) {
  hq::BlockGemmArgs p{};
  p.a = a;
  p.sa = sfa;
  p.b = b;
  p.sb = sfb;
  p.out = out;
  p.rows = rows;
  p.n = n;
  p.k = k;
  p.groups = groups;
  p.form = form;
  return p;
}

hq_status run_product(const char* what, void* stream, const hq::BlockGemmArgs& p, void* ws, uint64_t ws_bytes) {
  hq::DeviceInfo dev;
  const hq_status st = current_device(&dev);
  if (st != HQ_OK) return st;
  return launched(hq::launch_block_gemm((hipStream_t)stream, p, dev, ws, ws_bytes), what);
}

hq_status check_groups(const char* what, int32_t num_groups) {
  if (num_groups < 1 || num_groups > 1024)
    return fail(HQ_ERR_SHAPE, "%s: num_groups=%d must be in [1, 1024]", what, num_groups);
  return HQ_OK;
}

hq_status check_batch(const char* what, int64_t batch, int64_t m) {
  if (batch < 0 || batch > 65535) return fail(HQ_ERR_SHAPE, "%s: batch=%lld must be in [0, 65535]", what, (long long)batch);
  if (m < 0 || (batch > 0 && m > kI32 / batch))
    return fail(HQ_ERR_SHAPE, "%s: m=%lld: batch * m must be in [0, 2^31)", what, (long long)m);
  return HQ_OK;
}

// Checks common to the calls that walk a row map.
struct Map {
  int64_t tokens;
  int32_t topk;
  int64_t max_rows;
};
hq_status check_map(const char* what, const Map& m) {
  if (m.tokens < 0) return fail(HQ_ERR_SHAPE, "%s: num_tokens=%lld < 0", what, (long long)m.tokens);
  if (m.topk < 1 || m.topk > 64) return fail(HQ_ERR_SHAPE, "%s: topk=%d must be in [1, 64]", what, m.topk);
  if (m.tokens > kI32 / m.topk) return fail(HQ_ERR_SHAPE, "%s: num_tokens * topk must be < 2^31", what);
  if (m.max_rows < 0 || m.max_rows > kI32)
    return fail(HQ_ERR_SHAPE, "%s: max_rows=%lld must be in [0, 2^31)", what, (long long)m.max_rows);
  return HQ_OK;
}

hq_status check_pad(const char* what, const int32_t* group_end, const int32_t* counts, int32_t num_groups) {
  if ((group_end != nullptr) != (counts != nullptr))
    return fail(HQ_ERR_NULL, "%s: group_end and counts go together", what);
  if (group_end != nullptr) return check_groups(what, num_groups);
  return HQ_OK;
}

// The int32 tensors of those calls; any of them may be null.
hq_status check_index(const char* what, const int32_t* row_map, const int32_t* group_end, const int32_t* counts) {
  if (!aligned4(row_map) || !aligned4(group_end) || !aligned4(counts))
    return fail(HQ_ERR_ALIGN, "%s: row_map, group_end and counts must be 4-byte aligned", what);
  return HQ_OK;
}

// A width of h halves: 16-byte rows.
hq_status check_width(const char* what, int64_t h, int64_t step) {
  if (h <= 0 || h % step != 0 || h > kI32 / 16)
    return fail(HQ_ERR_SHAPE, "%s: hidden=%lld must be a positive multiple of %lld below 2^27", what, (long long)h,
                (long long)step);
  return HQ_OK;
}

// A launch's work items stay below the limit of one dimension.
hq_status check_grid(const char* what, int64_t workgroups, int threads) {
  if (workgroups > (hq::kMaxWorkItems - 1) / threads)
    return fail(HQ_ERR_SHAPE, "%s: problem too large: %lld workgroups of %d threads pass 2^32 work items", what,
                (long long)workgroups, threads);
  return HQ_OK;
}

}  // namespace

extern "C" {

hq_status hq_block_quant(void* stream, const uint16_t* x, int64_t batch, int64_t m, int64_t k, uint8_t* q, float* sf,
                         uint32_t flags) {
  const char* what = "hq_block_quant";
  if ((flags & ~(HQ_IN_FP16 | HQ_BLOCK_2D | HQ_TRANSPOSE)) != 0)
    return fail(HQ_ERR_MODE, "%s: unknown flags 0x%x", what, flags);
  hq_status st = check_batch(what, batch, m);
  if (st != HQ_OK) return st;
  if (k <= 0 || k % 32 != 0 || k > kI32)
    return fail(HQ_ERR_SHAPE, "%s: k=%lld must be a positive multiple of 32 below 2^31", what, (long long)k);
  if ((flags & HQ_TRANSPOSE) && m % 32 != 0)
    return fail(HQ_ERR_SHAPE, "%s: m=%lld must be a multiple of 32 with HQ_TRANSPOSE", what, (long long)m);
  const bool tiles = (flags & (HQ_BLOCK_2D | HQ_TRANSPOSE)) != 0;
  if ((st = check_grid(what, tiles ? hq::quant_tile_groups(batch, m, k) : hq::quant_row_groups(batch * m, k),
                       hq::kQuantThreads)) != HQ_OK)
    return st;
  if (batch == 0 || m == 0) return ok();
  if (!x || !q || !sf) return fail(HQ_ERR_NULL, "%s: x, q and sf are required", what);
  if (!aligned16(x) || !aligned16(q)) return fail(HQ_ERR_ALIGN, "%s: x and q must be 16-byte aligned", what);
  if (!aligned4(sf)) return fail(HQ_ERR_ALIGN, "%s: sf must be 4-byte aligned", what);
  hq::DeviceInfo dev;
  if ((st = current_device(&dev)) != HQ_OK) return st;
  return launched(hq::launch_block_quant((hipStream_t)stream, x, batch, m, k, q, sf, (flags & HQ_BLOCK_2D) != 0,
                                         (flags & HQ_TRANSPOSE) != 0, (flags & HQ_IN_FP16) != 0),
                  what);
}

hq_status hq_fused_swiglu_block_quant(void* stream, const uint16_t* x, int64_t rows, int64_t h,
                                      const int32_t* group_end, int32_t num_groups, uint8_t* q, float* sf,
                                      uint32_t flags) {
  const char* what = "hq_fused_swiglu_block_quant";
  if ((flags & ~HQ_IN_FP16) != 0) return fail(HQ_ERR_MODE, "%s: unknown flags 0x%x", what, flags);
  hq_status st;
  if (group_end != nullptr && (st = check_groups(what, num_groups)) != HQ_OK) return st;
  if (rows < 0 || rows > kI32) return fail(HQ_ERR_SHAPE, "%s: rows=%lld out of range", what, (long long)rows);
  if ((st = check_width(what, h, 32)) != HQ_OK) return st;
  if ((st = check_grid(what, hq::quant_row_groups(rows, h), hq::kQuantThreads)) != HQ_OK) return st;
  if (rows == 0) return ok();
  if (!x || !q || !sf) return fail(HQ_ERR_NULL, "%s: x, q and sf are required", what);
  if (!aligned16(x) || !aligned16(q)) return fail(HQ_ERR_ALIGN, "%s: x and q must be 16-byte aligned", what);
  if (!aligned4(sf) || !aligned4(group_end))
    return fail(HQ_ERR_ALIGN, "%s: sf and group_end must be 4-byte aligned", what);
  hq::DeviceInfo dev;
  if ((st = current_device(&dev)) != HQ_OK) return st;
  return launched(hq::launch_swiglu_block_quant((hipStream_t)stream, x, rows, h,
                                                group_end != nullptr ? group_end + num_groups - 1 : nullptr, q, sf,
                                                (flags & HQ_IN_FP16) != 0),
                  what);
}

hq_status hq_block_gemm(void* stream, uint32_t flags, const uint8_t* a, const float* sfa, const uint8_t* b,
                        const float* sfb, void* out, int64_t batch, int64_t m, int64_t n, int64_t k, void* workspace,
                        uint64_t workspace_bytes) {
  const char* what = "hq_block_gemm";
  hq_status st = check_batch(what, batch, m);
  if (st != HQ_OK) return st;
  hq::BlockGemmArgs p = product(a, sfa, b, sfb, out, batch * m, n, k, (int32_t)batch, hq::kUniform);
  p.slot_rows = m;
  bool noop;
  if ((st = check_product(what, flags, p, &noop)) != HQ_OK) return st;
  if (workspace_bytes > 0 && workspace == nullptr)
    return fail(HQ_ERR_NULL, "%s: workspace is NULL but workspace_bytes > 0", what);
  if (workspace != nullptr && !aligned16(workspace))
    return fail(HQ_ERR_ALIGN, "%s: workspace must be 16-byte aligned", what);
  if (noop) return ok();
  return run_product(what, stream, p, workspace, workspace_bytes);
}

hq_status hq_block_gemm_workspace_size(uint32_t flags, int64_t batch, int64_t m, int64_t n, int64_t k,
                                       uint64_t* bytes) {
  const char* what = "hq_block_gemm_workspace_size";
  if (bytes == nullptr) return fail(HQ_ERR_NULL, "%s: bytes is required", what);
  hq_status st = check_batch(what, batch, m);
  if (st != HQ_OK) return st;
  // the pointers only have to pass the checks: nothing is read
  uint8_t* any = reinterpret_cast<uint8_t*>(16);
  float* anyf = reinterpret_cast<float*>(any);
  hq::BlockGemmArgs p = product(any, anyf, any, anyf, any, batch * m, n, k, (int32_t)batch, hq::kUniform);
  p.slot_rows = m;
  bool noop;
  if ((st = check_product(what, flags, p, &noop)) != HQ_OK) return st;
  *bytes = 0;
  if (noop) return ok();
  hq::DeviceInfo dev;
  if ((st = current_device(&dev)) != HQ_OK) return st;
  *bytes = hq::block_gemm_workspace_bytes(p, dev);
  return ok();
}

hq_status hq_block_group_contiguous_gemm(void* stream, uint32_t flags, const uint8_t* a, const float* sfa,
                                         const uint8_t* b, const float* sfb, const int32_t* group_end,
                                         int32_t num_groups, void* out, int64_t m_total, int64_t n, int64_t k) {
  const char* what = "hq_block_group_contiguous_gemm";
  hq_status st = check_groups(what, num_groups);
  if (st != HQ_OK) return st;
  hq::BlockGemmArgs p = product(a, sfa, b, sfb, out, m_total, n, k, num_groups, hq::kContiguous);
  p.group_end = group_end;
  bool noop;
  if ((st = check_product(what, flags, p, &noop)) != HQ_OK) return st;
  if (noop) return ok();
  if (!group_end) return fail(HQ_ERR_NULL, "%s: group_end is required", what);
  if (!aligned4(group_end)) return fail(HQ_ERR_ALIGN, "%s: group_end must be 4-byte aligned", what);
  return run_product(what, stream, p, nullptr, 0);
}

hq_status hq_block_group_masked_gemm(void* stream, uint32_t flags, const uint8_t* a, const float* sfa,
                                     const uint8_t* b, const float* sfb, const int32_t* masked_m, int32_t num_groups,
                                     int64_t max_m_per_group, void* out, int64_t n, int64_t k) {
  const char* what = "hq_block_group_masked_gemm";
  hq_status st = check_groups(what, num_groups);
  if (st != HQ_OK) return st;
  if (max_m_per_group <= 0 || max_m_per_group > kI32 / num_groups)
    return fail(HQ_ERR_SHAPE, "%s: max_m_per_group=%lld must be > 0 and num_groups * max_m below 2^31", what,
                (long long)max_m_per_group);
  hq::BlockGemmArgs p =
      product(a, sfa, b, sfb, out, num_groups * max_m_per_group, n, k, num_groups, hq::kMasked);
  p.slot_rows = max_m_per_group;
  p.counts = masked_m;
  bool noop;
  if ((st = check_product(what, flags, p, &noop)) != HQ_OK) return st;
  if (noop) return ok();
  if (!masked_m) return fail(HQ_ERR_NULL, "%s: masked_m is required", what);
  if (!aligned4(masked_m)) return fail(HQ_ERR_ALIGN, "%s: masked_m must be 4-byte aligned", what);
  return run_product(what, stream, p, nullptr, 0);
}

hq_status hq_block_group_k_gemm(void* stream, uint32_t flags, const uint8_t* a, const float* sfa, const uint8_t* b,
                                const float* sfb, const int32_t* group_end, int32_t num_groups, void* out, int64_t m,
                                int64_t n, int64_t k_total) {
  const char* what = "hq_block_group_k_gemm";
  hq_status st = check_groups(what, num_groups);
  if (st != HQ_OK) return st;
  if (k_total < 0 || k_total % 128 != 0)
    return fail(HQ_ERR_SHAPE, "%s: k_total=%lld must be a non-negative multiple of 128", what, (long long)k_total);
  if (m < 0 || m > kI32 / num_groups)
    return fail(HQ_ERR_SHAPE, "%s: m=%lld: num_groups * m must be in [0, 2^31)", what, (long long)m);
  hq::BlockGemmArgs p = product(a, sfa, b, sfb, out, num_groups * m, n, k_total > 0 ? k_total : 128, num_groups,
                                hq::kGroupK);
  p.group_end = group_end;
  bool noop;
  if (k_total == 0) {       // every group's sum is empty: a and b are not read
    p.a = p.b = static_cast<const uint8_t*>(out);
    p.sa = p.sb = static_cast<const float*>(out);
  }
  if ((st = check_product(what, flags, p, &noop)) != HQ_OK) return st;
  if (noop) return ok();
  if (!group_end) return fail(HQ_ERR_NULL, "%s: group_end is required", what);
  if (!aligned4(group_end)) return fail(HQ_ERR_ALIGN, "%s: group_end must be 4-byte aligned", what);
  p.rows = m;
  p.k = k_total;
  p.nkb = (int32_t)(k_total / 128);
  return run_product(what, stream, p, nullptr, 0);
}

static hq_status sort_shape(const char* what, int64_t tokens, int32_t topk, int32_t num_experts, int32_t align) {
  hq_status st = check_map(what, Map{tokens, topk, 0});
  if (st != HQ_OK) return st;
  if (num_experts < 1 || num_experts > 1024)
    return fail(HQ_ERR_SHAPE, "%s: num_experts=%d must be in [1, 1024]", what, num_experts);
  if (align < 1 || align > 1024) return fail(HQ_ERR_SHAPE, "%s: align=%d must be in [1, 1024]", what, align);
  return HQ_OK;
}

// The most rows that the sorted pairs and their padding can take.
static int64_t sort_rows(int64_t pairs, int64_t experts, int64_t align) {
  return (pairs + (experts < pairs ? experts : pairs) * (align - 1)) / align * align;
}

hq_status hq_moe_sort_workspace_size(int64_t num_tokens, int32_t topk, int32_t num_experts, uint64_t* bytes) {
  const char* what = "hq_moe_sort_workspace_size";
  if (bytes == nullptr) return fail(HQ_ERR_NULL, "%s: bytes is required", what);
  const hq_status st = sort_shape(what, num_tokens, topk, num_experts, 1);
  if (st != HQ_OK) return st;
  *bytes = hq::moe_sort_workspace_bytes(num_tokens * topk, num_experts);
  return ok();
}

hq_status hq_moe_sort(void* stream, const int64_t* topk_ids, int64_t num_tokens, int32_t topk, int32_t num_experts,
                      int32_t align, int64_t max_rows, int32_t* row_map, int32_t* row_pair, int32_t* group_end,
                      int32_t* counts, void* workspace, uint64_t workspace_bytes) {
  const char* what = "hq_moe_sort";
  hq_status st = sort_shape(what, num_tokens, topk, num_experts, align);
  if (st != HQ_OK) return st;
  const int64_t pairs = num_tokens * topk;
  if (max_rows > kI32 || max_rows < sort_rows(pairs, num_experts, align))
    return fail(HQ_ERR_SHAPE, "%s: max_rows=%lld: %lld pairs of %d experts aligned to %d need up to %lld rows (below 2^31)",
                what, (long long)max_rows, (long long)pairs, num_experts, align,
                (long long)sort_rows(pairs, num_experts, align));
  if (!group_end || !counts || (pairs > 0 && (!topk_ids || !row_map)) || (max_rows > 0 && !row_pair))
    return fail(HQ_ERR_NULL, "%s: topk_ids, row_map, row_pair, group_end and counts are required", what);
  const uint64_t need = hq::moe_sort_workspace_bytes(pairs, num_experts);
  if (need > 0 && workspace == nullptr) return fail(HQ_ERR_NULL, "%s: this shape needs a workspace", what);
  if (workspace_bytes < need)
    return fail(HQ_ERR_SHAPE, "%s: workspace_bytes=%llu, this shape needs %llu", what,
                (unsigned long long)workspace_bytes, (unsigned long long)need);
  if (!aligned8(topk_ids)) return fail(HQ_ERR_ALIGN, "%s: topk_ids must be 8-byte aligned", what);
  if (!aligned4(row_map) || !aligned4(row_pair) || !aligned4(group_end) || !aligned4(counts) || !aligned4(workspace))
    return fail(HQ_ERR_ALIGN, "%s: row_map, row_pair, group_end, counts and the workspace must be 4-byte aligned", what);
  hq::DeviceInfo dev;
  if ((st = current_device(&dev)) != HQ_OK) return st;
  return launched(hq::launch_moe_sort((hipStream_t)stream, topk_ids, pairs, num_experts, align, max_rows, row_map,
                                      row_pair, group_end, counts, workspace),
                  what);
}

hq_status hq_moe_permute(void* stream, const uint8_t* x, int64_t num_tokens, int64_t row_bytes,
                         const int32_t* row_map, int32_t topk, const int32_t* group_end, const int32_t* counts,
                         int32_t num_groups, int64_t max_rows, uint8_t* out) {
  const char* what = "hq_moe_permute";
  hq_status st = check_map(what, Map{num_tokens, topk, max_rows});
  if (st != HQ_OK) return st;
  if ((st = check_pad(what, group_end, counts, num_groups)) != HQ_OK) return st;
  if (row_bytes <= 0 || row_bytes % 16 != 0 || row_bytes > kI32)
    return fail(HQ_ERR_SHAPE, "%s: row_bytes=%lld must be a positive multiple of 16 below 2^31", what,
                (long long)row_bytes);
  const hq::PadRows pad{group_end, counts, num_groups};
  if ((st = check_grid(what, hq::piece_groups(num_tokens, row_bytes, 1024) + hq::pad_groups(pad), hq::kMoeThreads)) !=
      HQ_OK)
    return st;
  if (max_rows == 0) return ok();
  if (!out || (num_tokens > 0 && (!x || !row_map))) return fail(HQ_ERR_NULL, "%s: x, row_map and out are required", what);
  if (!aligned16(x) || !aligned16(out)) return fail(HQ_ERR_ALIGN, "%s: x and out must be 16-byte aligned", what);
  if ((st = check_index(what, row_map, group_end, counts)) != HQ_OK) return st;
  hq::DeviceInfo dev;
  if ((st = current_device(&dev)) != HQ_OK) return st;
  return launched(hq::launch_moe_permute((hipStream_t)stream, x, num_tokens, row_bytes, row_map, topk, pad, max_rows,
                                         out),
                  what);
}

hq_status hq_moe_permute_block_quant(void* stream, const uint16_t* x, int64_t num_tokens, int64_t hidden,
                                     const int32_t* row_map, int32_t topk, const int32_t* group_end,
                                     const int32_t* counts, int32_t num_groups, int64_t max_rows, uint8_t* q,
                                     float* sf, uint32_t flags) {
  const char* what = "hq_moe_permute_block_quant";
  if ((flags & ~HQ_IN_FP16) != 0) return fail(HQ_ERR_MODE, "%s: unknown flags 0x%x", what, flags);
  hq_status st = check_map(what, Map{num_tokens, topk, max_rows});
  if (st != HQ_OK) return st;
  if ((st = check_pad(what, group_end, counts, num_groups)) != HQ_OK) return st;
  if ((st = check_width(what, hidden, 32)) != HQ_OK) return st;
  const hq::PadRows pad{group_end, counts, num_groups};
  if ((st = check_grid(what, hq::piece_groups(num_tokens, hidden, 1024) + hq::pad_groups(pad), hq::kMoeThreads)) !=
      HQ_OK)
    return st;
  if (max_rows == 0) return ok();
  if (!q || !sf || (num_tokens > 0 && (!x || !row_map)))
    return fail(HQ_ERR_NULL, "%s: x, row_map, q and sf are required", what);
  if (!aligned16(x) || !aligned16(q)) return fail(HQ_ERR_ALIGN, "%s: x and q must be 16-byte aligned", what);
  if (!aligned4(sf)) return fail(HQ_ERR_ALIGN, "%s: sf must be 4-byte aligned", what);
  if ((st = check_index(what, row_map, group_end, counts)) != HQ_OK) return st;
  hq::DeviceInfo dev;
  if ((st = current_device(&dev)) != HQ_OK) return st;
  return launched(hq::launch_moe_permute_block_quant((hipStream_t)stream, x, num_tokens, hidden, row_map, topk, pad,
                                                     max_rows, q, sf, (flags & HQ_IN_FP16) != 0),
                  what);
}

hq_status hq_moe_combine(void* stream, const uint16_t* y, int64_t num_tokens, int64_t hidden, const int32_t* row_map,
                         int32_t topk, const float* weights, int64_t max_rows, uint16_t* out, uint32_t flags) {
  const char* what = "hq_moe_combine";
  if ((flags & ~HQ_IN_FP16) != 0) return fail(HQ_ERR_MODE, "%s: unknown flags 0x%x", what, flags);
  hq_status st = check_map(what, Map{num_tokens, topk, max_rows});
  if (st != HQ_OK) return st;
  if ((st = check_width(what, hidden, 8)) != HQ_OK) return st;
  if ((st = check_grid(what, hq::piece_groups(num_tokens, hidden, 512), hq::kMoeThreads)) != HQ_OK) return st;
  if (num_tokens == 0) return ok();
  if (!out || !row_map || (max_rows > 0 && !y)) return fail(HQ_ERR_NULL, "%s: y, row_map and out are required", what);
  if (!aligned16(y) || !aligned16(out)) return fail(HQ_ERR_ALIGN, "%s: y and out must be 16-byte aligned", what);
  if (!aligned4(weights)) return fail(HQ_ERR_ALIGN, "%s: weights must be 4-byte aligned", what);
  if ((st = check_index(what, row_map, nullptr, nullptr)) != HQ_OK) return st;
  hq::DeviceInfo dev;
  if ((st = current_device(&dev)) != HQ_OK) return st;
  return launched(hq::launch_moe_combine((hipStream_t)stream, y, num_tokens, hidden, row_map, topk, weights, max_rows,
                                         out, (flags & HQ_IN_FP16) != 0),
                  what);
}

hq_status hq_moe_combine_backward(void* stream, const uint16_t* dout, const uint16_t* y, int64_t num_tokens,
                                  int64_t hidden, const int32_t* row_map, int32_t topk, const float* weights,
                                  const int32_t* group_end, const int32_t* counts, int32_t num_groups,
                                  int64_t max_rows, uint16_t* dy, float* dweights, uint32_t flags) {
  const char* what = "hq_moe_combine_backward";
  if ((flags & ~HQ_IN_FP16) != 0) return fail(HQ_ERR_MODE, "%s: unknown flags 0x%x", what, flags);
  hq_status st = check_map(what, Map{num_tokens, topk, max_rows});
  if (st != HQ_OK) return st;
  if ((st = check_pad(what, group_end, counts, num_groups)) != HQ_OK) return st;
  if ((st = check_width(what, hidden, 8)) != HQ_OK) return st;
  const hq::PadRows pad{group_end, counts, num_groups};
  if ((st = check_grid(what, num_tokens + hq::pad_groups(pad), 64 * hq::combine_bwd_waves(topk))) != HQ_OK) return st;
  if (num_tokens == 0 && (max_rows == 0 || group_end == nullptr)) return ok();
  if ((max_rows > 0 && (!dy || !y)) || (num_tokens > 0 && (!dout || !row_map || !weights || !dweights)))
    return fail(HQ_ERR_NULL, "%s: dout, y, row_map, weights, dy and dweights are required", what);
  if (!aligned16(dout) || !aligned16(y) || !aligned16(dy))
    return fail(HQ_ERR_ALIGN, "%s: dout, y and dy must be 16-byte aligned", what);
  if (!aligned4(weights) || !aligned4(dweights))
    return fail(HQ_ERR_ALIGN, "%s: weights and dweights must be 4-byte aligned", what);
  if ((st = check_index(what, row_map, group_end, counts)) != HQ_OK) return st;
  hq::DeviceInfo dev;
  if ((st = current_device(&dev)) != HQ_OK) return st;
  return launched(hq::launch_moe_combine_backward((hipStream_t)stream, dout, y, num_tokens, hidden, row_map, topk,
                                                  weights, pad, max_rows, dy, dweights, (flags & HQ_IN_FP16) != 0),
                  what);
}

}  // extern "C"
