// 16-bit products by expert: out[r] = a[r] b[g]^T (or a[r] b[g]) for the rows r
// of group g, and out[g] = sum over its rows of a[r]^T b[r].
#include "half_launch.hpp"

namespace hq {
namespace {

int plan_half(const HalfGemmArgs& p) {
  if (p.form == kGroupK) return p.rows >= 256 && p.n >= 256 ? kHalf256x256 : kHalf128x128;
  const int64_t per = p.form == kContiguous ? p.rows / p.groups : p.slot_rows;
  return per <= 64 ? kHalf64x128 : per <= 256 ? kHalf128x128 : kHalf256x256;
}

}  // namespace

hipError_t launch_half_gemm(hipStream_t s, const HalfGemmArgs& p, const DeviceInfo& dev) {
  const int tile = plan_half(p);
  if (p.form == kGroupK) return launch_half_tn(s, p, dev, tile);
  return p.b_t ? launch_half_nn(s, p, dev, tile) : launch_half_nt(s, p, dev, tile);
}

}  // namespace hq
