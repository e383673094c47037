// dma.hpp -- loads from a buffer straight into LDS, and the waits they need.
#pragma once

#include <stdint.h>

#include "common.hpp"

namespace is {

typedef unsigned uintx4 __attribute__((ext_vector_type(4)));

constexpr unsigned kOutside = 0xFFFFFFF0u;   // an offset outside every buffer: zeros

// A buffer of `bytes` at `at` (both alike in all lanes). An offset (unsigned) that is not inside reads zeros.
__device__ __forceinline__ uintx4 buffer_at(uint64_t at, unsigned bytes) {
  return uintx4{(unsigned)__builtin_amdgcn_readfirstlane((unsigned)at),
                (unsigned)__builtin_amdgcn_readfirstlane((unsigned)(at >> 32) & 0xffffu),
                (unsigned)__builtin_amdgcn_readfirstlane(bytes), (unsigned)kBufferFlags};
}

// N operations of 16 bytes per lane, operation i to dst + 1024 i + 16 lane of LDS.
// Written as instructions because the compiler takes the builtin for a store that
// any later LDS read may meet, and waits for it there; loads_left() is the wait.
// They have no output register, so nothing is open while they run. The s_nop 4 keeps
// a descriptor that a vector instruction brought to scalar registers (a spill) five
// wait states from its first use.
#define IS_LOAD16(O) "buffer_load_dwordx4 " O ", %1, 0 offen lds\n\t"
#define IS_NEXT "s_add_u32 m0, m0, 0x400\n\ts_nop 0\n\t"
template <int N>
__device__ __forceinline__ void load_lds16(uintx4 rs, unsigned dst, const unsigned *o) {
  if constexpr (N >= 4) {
    __asm__ volatile("s_mov_b32 m0, %0\n\ts_nop 4\n\t" IS_LOAD16("%2") IS_NEXT IS_LOAD16("%3") IS_NEXT IS_LOAD16("%4")
                         IS_NEXT IS_LOAD16("%5")
                     :
                     : "s"(dst), "s"(rs), "v"(o[0]), "v"(o[1]), "v"(o[2]), "v"(o[3])
                     : "memory", "scc");
    if constexpr (N > 4) load_lds16<N - 4>(rs, dst + 4096, o + 4);
  } else if constexpr (N >= 2) {
    __asm__ volatile("s_mov_b32 m0, %0\n\ts_nop 4\n\t" IS_LOAD16("%2") IS_NEXT IS_LOAD16("%3")
                     :
                     : "s"(dst), "s"(rs), "v"(o[0]), "v"(o[1])
                     : "memory", "scc");
    if constexpr (N > 2) load_lds16<N - 2>(rs, dst + 2048, o + 2);
  } else if constexpr (N == 1) {
    __asm__ volatile("s_mov_b32 m0, %0\n\ts_nop 4\n\t" IS_LOAD16("%2")
                     :
                     : "s"(dst), "s"(rs), "v"(o[0])
                     : "memory");
  }
}
#undef IS_LOAD16
#undef IS_NEXT

// One operation of 4 bytes per lane.
__device__ __forceinline__ void load_lds4(uintx4 rs, unsigned dst, unsigned off) {
  __asm__ volatile("s_mov_b32 m0, %0\n\ts_nop 4\n\tbuffer_load_dword %1, %2, 0 offen lds"
                   :
                   : "s"(dst), "v"(off), "s"(rs)
                   : "memory");
}

// Until at most N of this wave's vector-memory operations are outstanding.
template <int N>
__device__ __forceinline__ void loads_left() {
  __asm__ volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt(0x0F70 | (N & 15) | (N >> 4) << 14);
  __asm__ volatile("" ::: "memory");
}

}  // namespace is
