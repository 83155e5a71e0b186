// Copies from global memory straight into LDS (16 bytes a lane, lane-linear
// in LDS from the wave's LDS address).  Issued from inline assembly so that
// the compiler does not fold them into its own vmcnt bookkeeping; their
// completion is awaited explicitly (dma_wait), and read by other waves only
// behind a barrier.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace coli {

__device__ __forceinline__ uint32_t lds_addr(const char *p) {
  return (uint32_t)(uintptr_t)(const __attribute__((address_space(3))) char *)p;
}

// M0 holds the LDS address of lane 0's data (one wait state between the M0
// write and the load).
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"
__device__ __forceinline__ void dma16(uint32_t lds, const void *base, uint32_t off) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2" ::"s"(lds), "v"(off), "s"(base)
               : "memory", "m0");
}
__device__ __forceinline__ void dma16v(uint32_t lds, const void *addr) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, off" ::"s"(lds), "v"(addr)
               : "memory", "m0");
}
template <int N>
__device__ __forceinline__ void dma_wait() {
  asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}
#pragma clang diagnostic pop

}  // namespace coli
