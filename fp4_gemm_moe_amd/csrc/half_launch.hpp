// Host side of the tiled 16-bit GEMM: launches.
#pragma once

#include <atomic>

#include "half_plan.hpp"
#include "half_tiled.hpp"

namespace hq {

// One launch with the operands as the products have them: a and b K-minor (nt),
// b K-major outside (nn), both (tn, the form that sums over the groups' rows).
hipError_t launch_half_nt(hipStream_t s, const HalfGemmArgs& p, const DeviceInfo& dev, int tile);
hipError_t launch_half_nn(hipStream_t s, const HalfGemmArgs& p, const DeviceInfo& dev, int tile);
hipError_t launch_half_tn(hipStream_t s, const HalfGemmArgs& p, const DeviceInfo& dev, int tile);

namespace half {

// At most this many tiles (row forms know their counts on the device).
template <class C>
int64_t tile_count(const HalfGemmArgs& p) {
  const int64_t nt = (p.n + C::BN - 1) / C::BN;
  if (p.form == kGroupK) return (p.rows + C::BM - 1) / C::BM * nt * p.groups;
  if (p.form == kMasked) return (p.slot_rows + C::BM - 1) / C::BM * p.groups * nt;
  return (p.rows / C::BM + p.groups) * nt;
}

template <class C, bool AT, bool BT, bool F16>
hipError_t launch_one(hipStream_t s, const HalfGemmArgs& p, const DeviceInfo& dev) {
  // the dynamic-LDS attribute, once per device (setting it twice is harmless)
  static std::atomic<bool> set[64];
  const bool cached = dev.device >= 0 && dev.device < 64;
  if (!cached || !set[dev.device].load(std::memory_order_acquire)) {
    const hipError_t e = hipFuncSetAttribute((const void*)half_gemm_tiled<C, AT, BT, F16>,
                                             hipFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
    if (e != hipSuccess) return e;
    if (cached) set[dev.device].store(true, std::memory_order_release);
  }
  // one workgroup per compute unit; whole eighths, one for each XCD
  int64_t grid = (tile_count<C>(p) + 7) / 8 * 8;
  if (grid > dev.num_cus) grid = dev.num_cus;
  hipLaunchKernelGGL((half_gemm_tiled<C, AT, BT, F16>), dim3((unsigned)grid), dim3(C::THREADS), C::SMEM, s, p);
  return hipGetLastError();
}

template <class C, bool AT, bool BT>
hipError_t launch_type(hipStream_t s, const HalfGemmArgs& p, const DeviceInfo& dev) {
  return p.f16 ? launch_one<C, AT, BT, true>(s, p, dev) : launch_one<C, AT, BT, false>(s, p, dev);
}

// The tiles that plan_half has for the form: sums over the rows take two of them.
template <bool AT, bool BT>
hipError_t launch_tile(hipStream_t s, const HalfGemmArgs& p, const DeviceInfo& dev, int tile) {
  if (tile == kHalf256x256) return launch_type<Cfg<256, 256, 2, 2, 2>, AT, BT>(s, p, dev);
  if (tile == kHalf128x128) return launch_type<Cfg<128, 128, 2, 2, 4>, AT, BT>(s, p, dev);
  if constexpr (!AT) {
    if (tile == kHalf128x256) return launch_type<Cfg<128, 256, 2, 2, 2>, AT, BT>(s, p, dev);
    if (tile == kHalf64x128) return launch_type<Cfg<64, 128, 1, 4, 5>, AT, BT>(s, p, dev);
    if (tile == kHalf32x64) return launch_type<Cfg<32, 64, 1, 2, 9>, AT, BT>(s, p, dev);
  }
  return hipErrorInvalidValue;           // no such plan
}

}  // namespace half
}  // namespace hq
