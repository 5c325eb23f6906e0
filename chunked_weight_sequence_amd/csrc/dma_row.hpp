// Direct copies from global memory to LDS, several in a row.
#pragma once
#include <cstdint>

#include "dma.hpp"

namespace ttt {

// Direct copies (dma.hpp) in a row, 1 KB apart in LDS (m0 + 1024 I): the instruction's offset counts
// for the global address and the LDS address alike, so M0 is written once, by the first (I = 0), a wait
// state ahead. The I-th copy reads at sbase + voff + 1024 I.
template <int I>
__device__ __forceinline__ void dma16_at(uint32_t voff, const char* sbase, uint32_t m0) {
  if constexpr (I == 0)
    asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, %1" ::"v"(voff), "s"(sbase),
                 "s"(m0));
  else
    asm volatile("global_load_lds_dwordx4 %0, %1 offset:%2" ::"v"(voff), "s"(sbase), "n"(I * 1024));
}

}  // namespace ttt
