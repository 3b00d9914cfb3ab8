// Loads that go straight to LDS, and the waits that belong to them (gfx950).
//
// They are asm because the waits are counted by the kernels: the compiler would
// have to take every LDS read for one that may meet the newest load. What it
// does for its own instructions is therefore done here:
//  - An SGPR that the vector ALU has written (v_readlane, v_readfirstlane: the
//    words of a descriptor, the LDS address) may be read by a vector-memory
//    instruction five wait states later. The compiler counts none for asm, so
//    each load brings its own five: s_mov_b32 and s_nop 3.
//  - m0 needs one wait state after s_mov_b32, which those cover. It is a
//    reserved register: the compiler keeps no value in it, but sets it anew
//    before each use of its own (and refuses it in a list of clobbers).
//  - There is no register to be overwritten in flight; the address registers
//    are read at issue.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

namespace bsqd {

typedef uint32_t rsrc_words __attribute__((ext_vector_type(4)));

// A value that is the same in every lane, told to the compiler (it goes to a
// scalar register; descriptors and loop bounds made of it need no lane loops).
__device__ __forceinline__ int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }

__device__ __forceinline__ rsrc_words descriptor(const void* p, uint32_t bytes) {
  const uint64_t at = (uint64_t)p;
  return (rsrc_words){(uint32_t)uniform((int)(uint32_t)at), (uint32_t)uniform((int)(uint32_t)(at >> 32)) & 0xFFFFu,
                      (uint32_t)uniform((int)bytes), 0x00020000u};
}

// Where a lane's load goes. There is nothing to load where `there` is false (the
// same in every lane) or `mine` is: such a load is issued all the same, for the
// waits that count it, past the buffer's end. A raw buffer's range check is
// voff >= bytes - soff, in unsigned 32 bits, so a scalar offset that is itself
// past the end must not stand there: the difference would wrap and let any lane
// offset pass.
constexpr uint32_t kPastEnd = 0x80000000u;  // past every buffer that is read this way
struct BufferAt {
  uint32_t voff, soff;
};
__host__ __device__ constexpr BufferAt buffer_at(bool there, bool mine, uint32_t voff, uint32_t soff) {
  return {there && mine ? voff : kPastEnd, there ? soff : 0u};
}

// 64 lanes of SIZE bytes (4 or 16) each: lane l's at lds + SIZE l.
template <int SIZE>
__device__ __forceinline__ void load_to_lds(rsrc_words rsrc, uint32_t voff, uint32_t soff, uint32_t lds) {
  static_assert(SIZE == 4 || SIZE == 16, "sizes of the instruction");
  if constexpr (SIZE == 16)
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 3\n\tbuffer_load_dwordx4 %1, %2, %3 offen lds" ::"s"(lds), "v"(voff),
                 "s"(rsrc), "s"(soff)
                 : "memory");
  else
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 3\n\tbuffer_load_dword %1, %2, %3 offen lds" ::"s"(lds), "v"(voff),
                 "s"(rsrc), "s"(soff)
                 : "memory");
}

template <int SIZE>
__device__ __forceinline__ void load_to_lds(rsrc_words rsrc, BufferAt at, uint32_t lds) {
  load_to_lds<SIZE>(rsrc, at.voff, at.soff, lds);
}

template <int N>
__device__ __forceinline__ void wait_loads() {  // all but the N youngest
  asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}
__device__ __forceinline__ void wait_lds() { asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory"); }

// Workgroup barrier that completes this wave's LDS operations and leaves its
// loads in flight.
__device__ __forceinline__ void lds_barrier() { asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory"); }

__device__ __forceinline__ uint32_t lds_offset(const void* p) {
  return (uint32_t)uniform((int)(uint32_t)(uintptr_t)(__attribute__((address_space(3))) const void*)p);
}

}  // namespace bsqd
