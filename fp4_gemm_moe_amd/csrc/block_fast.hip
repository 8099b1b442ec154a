// Instantiations of the tiled block-128 FP8 GEMM on the FP8 matrix
// instructions: BF16 results, and FP32 partial sums of a K split that a BF16
// result is made of.
#include "block_launch.hpp"

namespace hq {
namespace {

// Partial sums are read again at once and are never streamed out.
template <class C>
hipError_t launch(hipStream_t s, const BlockGemmArgs& p, const DeviceInfo& dev, int policy) {
  using namespace blk;
  if (p.out_kind == kOutF32) return launch_one<C, kOutF32, kPolKeep>(s, p, dev);
  return launch_out<C, kOutBf16>(s, p, dev, policy);
}

}  // namespace

hipError_t launch_block_fast(hipStream_t s, const BlockGemmArgs& p, const DeviceInfo& dev, int tile, int policy) {
  using namespace blk;
  switch (tile) {
    case kTile256x256: return launch<Cfg<256, 256, 2, 4, 2, true>>(s, p, dev, policy);
    case kTile128x256: return launch<Cfg<128, 256, 2, 4, 3, true>>(s, p, dev, policy);
    case kTile128x128: return launch<Cfg<128, 128, 2, 2, 4, true>>(s, p, dev, policy);
    default: return launch<Cfg<64, 128, 2, 2, 5, true>>(s, p, dev, policy);
  }
}

}  // namespace hq
