// Host side of the tiled block-128 FP8 GEMM: tile shapes and launches.
#pragma once

#include <atomic>
#include <type_traits>

#include "block_tiled.hpp"

namespace hq {

// Tile shapes of the tiled kernel (rows x columns).
enum BlockTile : int { kTile256x256, kTile256x128, kTile128x256, kTile128x128, kTile64x128 };

hipError_t launch_block_fast(hipStream_t s, const BlockGemmArgs& p, const DeviceInfo& dev, int tile, bool nt);
hipError_t launch_block_exact(hipStream_t s, const BlockGemmArgs& p, const DeviceInfo& dev, int tile, bool nt);

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

template <class C, int OUT, bool NT>
hipError_t launch_one(hipStream_t s, const BlockGemmArgs& p, const DeviceInfo& dev) {
  // the dynamic-LDS attribute, once per device (setting it twice is harmless)
  static std::atomic<bool> set[64];
  const bool cached = dev.device >= 0 && dev.device < 64;
  if (!cached || !set[dev.device].load(std::memory_order_acquire)) {
    const hipError_t e = hipFuncSetAttribute((const void*)block_gemm_tiled<C, OUT, NT>,
                                             hipFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
    if (e != hipSuccess) return e;
    if (cached) set[dev.device].store(true, std::memory_order_release);
  }
  // one workgroup per compute unit; whole eighths, one for each XCD
  int64_t grid = (tile_count<C>(p) + 7) / 8 * 8;
  if (grid > dev.num_cus) grid = dev.num_cus;
  hipLaunchKernelGGL((block_gemm_tiled<C, OUT, NT>), dim3((unsigned)grid), dim3(C::THREADS), C::SMEM, s, p);
  return hipGetLastError();
}

// The instantiation for p's output among OUTS.
template <class C, int... OUTS>
hipError_t launch_out(hipStream_t s, const BlockGemmArgs& p, const DeviceInfo& dev, bool nt) {
  hipError_t e = hipErrorInvalidValue;
  (void)((p.out_kind == OUTS
              ? (e = nt ? launch_one<C, OUTS, true>(s, p, dev) : launch_one<C, OUTS, false>(s, p, dev), true)
              : false) ||
         ...);
  return e;
}

}  // namespace blk
}  // namespace hq
