// Instantiations of the tiled 16-bit GEMM: both operands K-minor.
#include "half_launch.hpp"

namespace hq {

hipError_t launch_half_nt(hipStream_t s, const HalfGemmArgs& p, const DeviceInfo& dev, int tile) {
  return half::launch_tile<false, false>(s, p, dev, tile);
}

}  // namespace hq
