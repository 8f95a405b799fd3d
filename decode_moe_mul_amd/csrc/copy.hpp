// Internal header: copies from memory to LDS that pass no registers.
#pragma once
#include "common.hpp"

namespace qmoe {

// a block-uniform address in scalar registers
QMOE_D const uint8_t* uniform(const uint8_t* p) {
  const uint64_t a = (uint64_t)p;
  const uint32_t lo = __builtin_amdgcn_readfirstlane((int)(uint32_t)a);
  const uint32_t hi = __builtin_amdgcn_readfirstlane((int)(uint32_t)(a >> 32));
  return (const uint8_t*)((uint64_t)hi << 32 | lo);
}

// 16 bytes a lane from base + off to LDS address lds + 16 * lane.  It has no
// output register; its completion is counted with the vector loads, in order,
// and waited for by wait_copies before the barrier that hands the data over.
// The compiler does not count it: its own waits for vector loads can only be
// longer than needed.  m0 is declared as written, so that no value of the
// compiler's own is taken to survive there (its warning that m0 is one of its
// reserved registers is expected).
QMOE_D void copy_to_lds(uint32_t lds, const uint8_t* base, uint32_t off) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2"
               :
               : "s"(__builtin_amdgcn_readfirstlane((int)lds)), "v"(off), "s"(base)
               : "m0", "memory");
}
QMOE_D void wait_copies() { asm volatile("s_waitcnt vmcnt(0)" ::: "memory"); }

}  // namespace qmoe
