// Instantiations of the tiled 16-bit GEMM: b with K outside.
#include "half_launch.hpp"

namespace hq {

hipError_t launch_half_nn(hipStream_t s, const HalfGemmArgs& p, const DeviceInfo& dev, int tile) {
  return half::launch_tile<false, true>(s, p, dev, tile);
}

}  // namespace hq
