// Pieces shared by the tiled kernels that load operands straight into LDS:
// uniform values, buffer descriptors, the loads, waits and the barrier.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace hq {
namespace blk {

__device__ __forceinline__ uint32_t ufirst(uint32_t v) { return __builtin_amdgcn_readfirstlane(v); }
__device__ __forceinline__ int64_t ufirst64(int64_t v) {
  const uint64_t u = (uint64_t)v;
  return (int64_t)(((uint64_t)ufirst((uint32_t)(u >> 32)) << 32) | ufirst((uint32_t)u));
}

// A pointer that is the same in every lane, which the compiler cannot prove.
template <class T>
__device__ __forceinline__ const T* uniform(const T* p) {
  return reinterpret_cast<const T*>(ufirst64((int64_t)(uintptr_t)p));
}

// Raw buffer descriptor over [base, base + bytes).  A tile's operands take
// less than 2^31 bytes, so an offset with bit 31 set lies outside.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t rsrc(const void* base, uint32_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), (short)0, (int)bytes, 0x00020000);
}

// Direct-to-LDS buffer loads of 16 / 4 bytes a lane (zeros when out of range)
// at voff + soff: lane j's result lands at LDS address lds + j * size.  In
// inline assembly, so that the compiler adds no waits of its own; the kernel
// waits on the vector-memory counter and a barrier before a stage is read.  m0
// is set inside each statement and used by nothing else; the load needs one
// wait state after that, which the compiler does not add inside a statement.
__device__ __forceinline__ void dma16(__amdgpu_buffer_rsrc_t r, uint32_t voff, uint32_t soff, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %3\n\ts_nop 0\n\tbuffer_load_dwordx4 %0, %1, %2 offen lds"
               ::"v"(voff), "s"(r), "s"(soff), "s"(lds) : "memory");
}
// The same for bytes that one workgroup reads once (non-temporal policy).
__device__ __forceinline__ void dma16nt(__amdgpu_buffer_rsrc_t r, uint32_t voff, uint32_t soff, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %3\n\ts_nop 0\n\tbuffer_load_dwordx4 %0, %1, %2 offen nt lds"
               ::"v"(voff), "s"(r), "s"(soff), "s"(lds) : "memory");
}
__device__ __forceinline__ void dma4(__amdgpu_buffer_rsrc_t r, uint32_t voff, uint32_t soff, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %3\n\ts_nop 0\n\tbuffer_load_dword %0, %1, %2 offen lds"
               ::"v"(voff), "s"(r), "s"(soff), "s"(lds) : "memory");
}

// The same from each lane's own address.
__device__ __forceinline__ void dma16_at(const void* p, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %1\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, off" ::"v"(p), "s"(lds) : "memory");
}

template <int N>
__device__ __forceinline__ void wait_vm() {
  asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}

// Workgroup barrier without a fence: the waits above order the LDS traffic.
__device__ __forceinline__ void bar() {
  __builtin_amdgcn_sched_barrier(0);
  __builtin_amdgcn_s_barrier();
  __builtin_amdgcn_sched_barrier(0);
}

}  // namespace blk
}  // namespace hq
