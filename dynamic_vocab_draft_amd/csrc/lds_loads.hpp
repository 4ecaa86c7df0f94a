// Loads from memory straight into LDS, and the waits that count them.
#pragma once
#include "rows.hpp"

namespace {

// 16 bytes a lane from a buffer straight into LDS at byte `lds` (the same
// for the wave) + 16 * lane.  The compiler does not count these loads: the
// waits below do.  m0 holds the LDS address.  The compiler does not see a
// memory instruction here either, so the asm keeps the distances itself: the
// move and the no-ops are the five wait states from a vector instruction that
// wrote an SGPR (v_readlane, as for a spilled one) to a memory instruction that
// reads it, and more than the one from the move to the load.  m0 is a register
// that the compiler reserves and writes before each use of its own, so it warns
// of the clobber, which tells it that the value is gone.
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"
__device__ __forceinline__ void load_to_lds(u32x4 rsrc, uint32_t voff, uint32_t soff, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %3\n\ts_nop 3\n\tbuffer_load_dwordx4 %0, %1, %2 offen lds"
               :
               : "v"(voff), "s"(rsrc), "s"(soff), "s"(lds)
               : "memory", "m0");
}

// The same for bytes that are read once: the caches need not keep them.
__device__ __forceinline__ void load_to_lds_once(u32x4 rsrc, uint32_t voff, uint32_t soff, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %3\n\ts_nop 3\n\tbuffer_load_dwordx4 %0, %1, %2 offen nt lds"
               :
               : "v"(voff), "s"(rsrc), "s"(soff), "s"(lds)
               : "memory", "m0");
}

// The same for four bytes a lane.
__device__ __forceinline__ void load_word_to_lds(u32x4 rsrc, uint32_t voff, uint32_t soff, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %3\n\ts_nop 3\n\tbuffer_load_dword %0, %1, %2 offen lds"
               :
               : "v"(voff), "s"(rsrc), "s"(soff), "s"(lds)
               : "memory", "m0");
}

#pragma clang diagnostic pop

__device__ __forceinline__ u32x4 buffer_of(const void* p, uint32_t bytes) {
  const uint64_t a = (uint64_t)p;
  return u32x4{(uint32_t)a, (uint32_t)(a >> 32) & 0xFFFFu, bytes, 0x00027000u};
}

template <int N>
__device__ __forceinline__ void wait_loads() {
  asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}

__device__ __forceinline__ uint32_t lds_offset(const void* p) {
  return (uint32_t)(uintptr_t)(const __attribute__((address_space(3))) char*)p;
}

}  // namespace
