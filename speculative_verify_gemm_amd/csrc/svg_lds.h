// Loads that go straight into LDS, and the waits that belong to them.
#pragma once
#include "svg_device.h"

// All but the last N loads of this wave have arrived, and everything it has read from LDS.
template <int N>
SVG_DEV void wait_loads() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt(0x0070 | (N & 15) | ((N >> 4) << 14));  // vmcnt(N) lgkmcnt(0)
  asm volatile("" ::: "memory");
}
SVG_DEV void barrier() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}
// 1 KiB from global memory at `from` (lane16: this lane's 16 bytes) straight into LDS at byte `to`; both the same for the
// wave.  In asm: the compiler would wait for all of them before it reads any LDS; here wait_loads() and the
// barrier say what has arrived.  m0 is declared: a value that the compiler puts there for itself is set anew behind this
// (the register is never allocated, of which it warns).
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"
SVG_DEV void load_to_lds(const char* from, u32 lane16, u32 to) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2"
               ::"s"(__builtin_amdgcn_readfirstlane((int)to)), "v"(lane16), "s"(from) : "memory", "m0");
}
#pragma clang diagnostic pop
// Bytes of LDS before p.
SVG_DEV u32 lds_at(const char* p) { return (u32)(uintptr_t)(const __attribute__((address_space(3))) char*)p; }
