// Tiles in LDS (gfx950): asynchronous loads to it, counted waits, and the
// swizzle of 64-byte rows, shared by the matrix kernels.
#pragma once

#include "block_device.h"

namespace block {

typedef __attribute__((address_space(3))) void lds_void;

// Global -> LDS, 16 bytes per lane: lane l's bytes land at lds + 16 l. Inline
// assembly, so that the compiler does not wait for every load in flight
// before each LDS read (it cannot tell the stages apart); the kernel's own
// vmcnt waits order them, and the volatile barriers below keep the LDS reads
// on their side.
__device__ __forceinline__ void dma16(const char* base, uint32_t off, uint32_t lds) {
  asm volatile("s_nop 0\n\tglobal_load_lds_dwordx4 %0, %1" : : "v"(off), "s"(base), "{m0}"(lds));
}
__device__ __forceinline__ void dma16(const char* addr, uint32_t lds) {
  asm volatile("s_nop 0\n\tglobal_load_lds_dwordx4 %0, off" : : "v"(addr), "{m0}"(lds));
}

// The same for what no other block reads: past the caches.
__device__ __forceinline__ void dma16_once(const char* addr, uint32_t lds) {
  asm volatile("s_nop 0\n\tglobal_load_lds_dwordx4 %0, off nt" : : "v"(addr), "{m0}"(lds));
}

__device__ __forceinline__ u32x4 lds_b128(uint32_t addr) {
  return *(const __attribute__((address_space(3))) u32x4*)(uintptr_t)addr;
}

// Wait until at most Vm of this wave's loads are in flight and at most Lgkm
// LDS reads are outstanding, then meet the block.
template <int Vm, int Lgkm>
__device__ __forceinline__ void wait_barrier() {
  static_assert(Vm >= 0 && Vm < 64 && Lgkm >= 0 && Lgkm < 16, "counter range");
  asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(%1)\n\ts_barrier" : : "n"(Vm), "n"(Lgkm) : "memory");
}

// Where the 16-byte piece c of a 64-byte row r sits: at c ^ swizzle(r >> 2).
__device__ __forceinline__ int swizzle(int r4) { return ((r4 ^ (r4 >> 1)) & 1) << 1 | ((r4 >> 1) & 1); }

}  // namespace block
