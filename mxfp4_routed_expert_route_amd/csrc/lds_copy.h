// Loads that write LDS themselves, and the waits and barriers that go with them.
#pragma once
#include "device.h"

namespace moe {

// 16 bytes a lane from `from` to LDS address lds + 16 * lane.  In assembly so that the compiler, which
// cannot tell one step's LDS from another's, does not wait for all copies before every LDS read;
// wait_copies counts them.  It writes no register: the LDS address is an operand in m0, which the
// compiler sets (the nop is the cycle between that and its use).
__device__ __forceinline__ void copy16_global(const void* from, uint32_t lds) {
  asm volatile("s_nop 0\n\tglobal_load_lds_dwordx4 %0, off" :: "v"(from), "{m0}"(lds) : "memory");
}
// Until at most kLeft of the wavefront's loads are on their way.
template <int kLeft>
__device__ __forceinline__ void wait_copies() {
  static_assert(kLeft < 64, "the counter's range");
  // vmcnt in bits 3:0 and 15:14, the other counters at their maximum (no wait)
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt((kLeft & 15) | ((kLeft >> 4) << 14) | 0x0F70);
  asm volatile("" ::: "memory");
}
__device__ __forceinline__ void wait_lds() { asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory"); }
__device__ __forceinline__ void barrier() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

}  // namespace moe
