// Instantiations of the tiled 16-bit GEMM: both operands with K outside (sums over the groups' rows).
#include "half_launch.hpp"

namespace hq {

hipError_t launch_half_tn(hipStream_t s, const HalfGemmArgs& p, const DeviceInfo& dev, int tile) {
  return half::launch_tile<true, true>(s, p, dev, tile);
}

}  // namespace hq
