// Direct loads from global memory to LDS (global_load_lds_*): lane l's bytes go
// to LDS address lds + 16 l (dwordx4) or lds + 4 l (dword), lds the same in every
// lane (in M0).  Written out rather than through the compiler builtin, whose wait
// insertion loses track of which buffer a pending load writes at a loop head and
// drains every load in flight.  The instruction has no register result, so no
// register can be overwritten by a load in flight; the kernels order LDS reads
// after it by explicit vmcnt waits.  M0 is an operand, so the compiler writes and
// tracks it.
//
// The hardware leaves two waits on this path to software, and the compiler adds
// none around inline assembly: one wait state between a scalar write of M0 and the
// load, five between a vector instruction's write of a scalar register (a uniform
// base may come from v_readfirstlane) and a memory instruction that reads it.
// The asm blocks hold them, whatever the compiler schedules before: a scalar copy of
// the base (the hardware waits for its source, and for a scalar write before the
// load) is the state behind M0 at the same time; without a base an s_nop is.  (With
// s_nop 4 in place of the copy, 2048 x 17408 x 5120: mx_linear_w4a4 162 us instead of
// 156.5, the W4A16 prefill 366 instead of 355.)
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace nvfp4 {

// The LDS byte address of p.
__device__ __forceinline__ uint32_t lds_addr(const void* p) {
  return (uint32_t)(uintptr_t)(__attribute__((address_space(3))) const void*)p;
}

// A pointer that is the same in every lane, in scalar registers (readfirstlane
// returns int: widened through uint32_t, never by sign extension).
template <typename T>
__device__ __forceinline__ const T* uniform_ptr(const T* p) {
  const uint64_t b = (uint64_t)(uintptr_t)p;
  return reinterpret_cast<const T*>(((uint64_t)(uint32_t)__builtin_amdgcn_readfirstlane((uint32_t)(b >> 32)) << 32) |
                                    (uint64_t)(uint32_t)__builtin_amdgcn_readfirstlane((uint32_t)b));
}

// From a uniform base and a byte offset per lane.
__device__ __forceinline__ void lds_dma16(const void* base, uint32_t off, uint32_t lds) {
  const uint32_t m0 = __builtin_amdgcn_readfirstlane(lds);
  uint64_t b;
  asm volatile("s_mov_b64 %0, %2\n\tglobal_load_lds_dwordx4 %1, %0"
               : "=&s"(b)
               : "v"(off), "s"(uniform_ptr((const char*)base)), "{m0}"(m0)
               : "memory");
}
__device__ __forceinline__ void lds_dma4(const void* base, uint32_t off, uint32_t lds) {
  const uint32_t m0 = __builtin_amdgcn_readfirstlane(lds);
  uint64_t b;
  asm volatile("s_mov_b64 %0, %2\n\tglobal_load_lds_dword %1, %0"
               : "=&s"(b)
               : "v"(off), "s"(uniform_ptr((const char*)base)), "{m0}"(m0)
               : "memory");
}

// From each lane's own address; _nt: with the nontemporal hint.
__device__ __forceinline__ void lds_dma16(const void* src, uint32_t lds) {
  const uint32_t m0 = __builtin_amdgcn_readfirstlane(lds);
  asm volatile("s_nop 0\n\tglobal_load_lds_dwordx4 %0, off" ::"v"(src), "{m0}"(m0) : "memory");
}
__device__ __forceinline__ void lds_dma16_nt(const void* src, uint32_t lds) {
  const uint32_t m0 = __builtin_amdgcn_readfirstlane(lds);
  asm volatile("s_nop 0\n\tglobal_load_lds_dwordx4 %0, off nt" ::"v"(src), "{m0}"(m0) : "memory");
}
__device__ __forceinline__ void lds_dma4(const void* src, uint32_t lds) {
  const uint32_t m0 = __builtin_amdgcn_readfirstlane(lds);
  asm volatile("s_nop 0\n\tglobal_load_lds_dword %0, off" ::"v"(src), "{m0}"(m0) : "memory");
}

}  // namespace nvfp4
