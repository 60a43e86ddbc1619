// Loads from global memory straight to LDS, and the barrier behind them.
#pragma once

#include <stdint.h>

#include <hip/hip_runtime.h>

namespace sv {

// A value that all lanes hold alike, in scalar registers.
__device__ __forceinline__ long long uniform(long long x) {
  const uint32_t lo = __builtin_amdgcn_readfirstlane((uint32_t)x);
  const uint32_t hi = __builtin_amdgcn_readfirstlane((uint32_t)((unsigned long long)x >> 32));
  return (long long)((unsigned long long)hi << 32 | lo);
}

// Loads from global memory to LDS at `to` (uniform) + 16 (4) * lane, by the active lanes.  In
// assembly because the compiler would wait for them before every LDS read it cannot tell apart; the
// kernel waits where it has to (tile_barrier).  No vector register is written; m0, which holds the
// LDS address, is declared (it is a reserved register, never kept across a statement, hence the
// compiler's warning), and needs one wait state before the load.
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"
__device__ __forceinline__ void load_to_lds(const char* from, uint32_t to) {
  asm volatile("s_mov_b32 m0, %1\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, off"
               :
               : "v"(from), "s"(__builtin_amdgcn_readfirstlane(to))
               : "memory", "m0");
}

// The same by those of the active lanes that are in `lanes` (uniform): a condition without a
// branch.  The execution mask is put back as it was.
__device__ __forceinline__ void load_to_lds(const char* from, uint32_t to,
                                            unsigned long long lanes) {
  unsigned long long active;
  asm volatile("s_mov_b32 m0, %2\n\ts_and_saveexec_b64 %0, %3\n\t"
               "global_load_lds_dwordx4 %1, off\n\ts_mov_b64 exec, %0"
               : "=&s"(active)
               : "v"(from), "s"(__builtin_amdgcn_readfirstlane(to)), "s"(uniform(lanes))
               : "memory", "m0", "scc");
}
#pragma clang diagnostic pop

// Waits for this wave's loads to LDS, then for the other waves'.
__device__ __forceinline__ void tile_barrier() {
  asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
}

}  // namespace sv
