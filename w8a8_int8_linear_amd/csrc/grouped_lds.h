// LDS transfers, fragment reads, waits and barriers of the grouped linears'
// kernels.
#pragma once
#include "grouped.h"

namespace convrot {
namespace {

typedef __attribute__((address_space(3))) void* lds_ptr_t;

// One 16-byte-per-lane global -> LDS transfer: lane l's bytes land at lds + 16 l.
__device__ __forceinline__ void dma16(const uint8_t* g, uint8_t* lds) {
#if defined(__HIP_DEVICE_COMPILE__)
  __builtin_amdgcn_global_load_lds(g, (lds_ptr_t)lds, 16, 0, 0);
#endif
}
// 16-byte LDS read in program order; the register is only safe to use past
// wait_lds() and landed().
template <int OFF>
__device__ __forceinline__ void lds_read16(i32x4& r, uint32_t addr) {
#if defined(__HIP_DEVICE_COMPILE__)
  asm volatile("ds_read_b128 %0, %1 offset:%2" : "=v"(r) : "v"(addr), "i"(OFF) : "memory");
#endif
}
// No instruction: uses of r stay behind the wait in front of this point.
__device__ __forceinline__ void landed(i32x4& r) {
#if defined(__HIP_DEVICE_COMPILE__)
  asm volatile("" : "+v"(r));
#endif
}
// No instruction: the compiler knows nothing of v's value past this point.
__device__ __forceinline__ void opaque(int& v) {
#if defined(__HIP_DEVICE_COMPILE__)
  asm volatile("" : "+v"(v));
#endif
}
__device__ __forceinline__ void wait_lds() {
#if defined(__HIP_DEVICE_COMPILE__)
  __builtin_amdgcn_s_waitcnt(0xC07F);  // lgkmcnt(0)
#endif
}
// At most N of this wave's vector-memory operations outstanding.
template <int N>
__device__ __forceinline__ void wait_vm() {
#if defined(__HIP_DEVICE_COMPILE__)
  static_assert(N >= 0 && N < 64, "vmcnt has 6 bits: [3:0] and [15:14]");
  __builtin_amdgcn_s_waitcnt((N & 15) | ((N >> 4) << 14) | (7 << 4) | (15 << 8));
#endif
}
// A wavefront's own LDS writes are visible to all its lanes past this point (its
// LDS operations complete in order; the compiler keeps them so).
__device__ __forceinline__ void wave_sync() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}
// Workgroup barrier without a fence: callers wait for what they need.
__device__ __forceinline__ void barrier() {
#if defined(__HIP_DEVICE_COMPILE__)
  __builtin_amdgcn_sched_barrier(0);
  __builtin_amdgcn_s_barrier();
  __builtin_amdgcn_sched_barrier(0);
#endif
}
template <int N, int I = 0, typename F>
__device__ __forceinline__ void static_for(F&& f) {
  if constexpr (I < N) {
    f(std::integral_constant<int, I>{});
    static_for<N, I + 1>(f);
  }
}

}  // namespace
}  // namespace convrot
