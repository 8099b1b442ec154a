// Host side of the tiled block-128 FP8 GEMM: launches.
#pragma once

#include <atomic>
#include <type_traits>

#include "block_plan.hpp"
#include "block_tiled.hpp"

namespace hq {

hipError_t launch_block_fast(hipStream_t s, const BlockGemmArgs& p, const DeviceInfo& dev, int tile, int policy);
hipError_t launch_block_exact(hipStream_t s, const BlockGemmArgs& p, const DeviceInfo& dev, int tile, int policy);

namespace blk {

// At most this many tiles (grouped row forms know their counts on the device).
template <class C>
int64_t tile_count(const BlockGemmArgs& p) {
  const int64_t nt = (p.n + C::BN - 1) / C::BN;
  auto up = [](int64_t r) { return (r + C::BM - 1) / C::BM; };
  if (p.form == kUniform) return up(p.slot_rows) * p.groups * nt * p.slices;
  if (p.form == kGroupK) return up(p.rows) * nt * p.groups;
  if (p.form == kMasked) return up(p.slot_rows) * p.groups * nt;
  return (p.rows / C::BM + p.groups) * nt;
}

template <class C, int OUT, int POL>
hipError_t launch_one(hipStream_t s, const BlockGemmArgs& p, const DeviceInfo& dev) {
  // the dynamic-LDS attribute, once per device (setting it twice is harmless)
  static std::atomic<bool> set[64];
  const bool cached = dev.device >= 0 && dev.device < 64;
  if (!cached || !set[dev.device].load(std::memory_order_acquire)) {
    const hipError_t e = hipFuncSetAttribute((const void*)block_gemm_tiled<C, OUT, POL>,
                                             hipFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
    if (e != hipSuccess) return e;
    if (cached) set[dev.device].store(true, std::memory_order_release);
  }
  // one workgroup per compute unit; whole eighths, one for each XCD
  int64_t grid = (tile_count<C>(p) + 7) / 8 * 8;
  if (grid > dev.num_cus) grid = dev.num_cus;
  hipLaunchKernelGGL((block_gemm_tiled<C, OUT, POL>), dim3((unsigned)grid), dim3(C::THREADS), C::SMEM, s, p);
  return hipGetLastError();
}

// The instantiation for the policy, and for p's output among OUTS.
template <class C, int OUT>
hipError_t launch_policy(hipStream_t s, const BlockGemmArgs& p, const DeviceInfo& dev, int policy) {
  if (policy == kPolStreamAll) return launch_one<C, OUT, kPolStreamAll>(s, p, dev);
  if (policy == kPolStreamOut) return launch_one<C, OUT, kPolStreamOut>(s, p, dev);
  return launch_one<C, OUT, kPolKeep>(s, p, dev);
}
template <class C, int... OUTS>
hipError_t launch_out(hipStream_t s, const BlockGemmArgs& p, const DeviceInfo& dev, int policy) {
  hipError_t e = hipErrorInvalidValue;
  (void)((p.out_kind == OUTS ? (e = launch_policy<C, OUTS>(s, p, dev, policy), true) : false) || ...);
  return e;
}

}  // namespace blk
}  // namespace hq
