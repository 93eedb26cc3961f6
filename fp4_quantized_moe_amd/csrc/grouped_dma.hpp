// Global-memory-to-LDS DMA of the MXFP4 and gated grouped kernels: dma.hpp's
// instructions and waits, for LDS addresses that the compiler does not know to
// be the same in all lanes (of a stage in turn, carried through loops): M0
// takes the first lane's.
#pragma once

#include "dma.hpp"

namespace quads {

__device__ __forceinline__ uint32_t lds_address(void *lds_base) {
  return __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(reinterpret_cast<uintptr_t>((lds_t *)lds_base)));
}

#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"
__device__ __forceinline__ void dma_wave(const void *g, void *lds_base, int bytes) {
  if (bytes == 16)
    asm volatile("s_mov_b32 m0, %1\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, off" ::"v"(g), "s"(lds_address(lds_base))
                 : "memory", "m0");
  else
    asm volatile("s_mov_b32 m0, %1\n\ts_nop 0\n\tglobal_load_lds_dword %0, off" ::"v"(g), "s"(lds_address(lds_base))
                 : "memory", "m0");
}
// 16 bytes a lane that the kernel does not come back to: their lines are the
// first to leave the caches.
__device__ __forceinline__ void dma_wave_once(const void *g, void *lds_base) {
  asm volatile("s_mov_b32 m0, %1\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, off nt" ::"v"(g), "s"(lds_address(lds_base))
               : "memory", "m0");
}
#pragma clang diagnostic pop

}  // namespace quads
