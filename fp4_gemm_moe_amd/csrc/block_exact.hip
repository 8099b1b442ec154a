// Instantiations of the tiled block-128 FP8 GEMM through FP16 operands: full
// FP32 sums, for FP16 and FP32 results and for short K.
#include "block_launch.hpp"

namespace hq {

hipError_t launch_block_exact(hipStream_t s, const BlockGemmArgs& p, const DeviceInfo& dev, int tile, int policy) {
  using namespace blk;
  if (tile == kTile128x128)
    return launch_out<Cfg<128, 128, 2, 2, 4, false>, kOutBf16, kOutF16, kOutF32, kOutF32Add>(s, p, dev, policy);
  if (tile == kTile256x128)
    return launch_out<Cfg<256, 128, 4, 2, 3, false>, kOutBf16, kOutF16, kOutF32, kOutF32Add>(s, p, dev, policy);
  return launch_out<Cfg<64, 128, 2, 2, 5, false>, kOutBf16, kOutF16, kOutF32, kOutF32Add>(s, p, dev, policy);
}

}  // namespace hq
