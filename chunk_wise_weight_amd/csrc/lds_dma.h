// Loads that go from memory straight into LDS, as instructions the compiler
// does not track: 16 (4) bytes per lane, lane l landing at the LDS address in
// M0 + 16 l (4 l).
//
// The compiler takes an LDS load of its own for a pending write to all of LDS,
// and before a transposing read (ds_read_b64_tr_b16) it waits for every one in
// flight. Untracked, the loads are ordered by a kernel's counted waits and
// barriers alone. They have no register outputs. M0 is the compiler's register:
// the block saves it in a scalar register of its own and puts it back. One wait
// state must pass between the write of M0 and the load that reads it, which the
// compiler counts for its own loads and the block for its.
#pragma once

#include <hip/hip_runtime.h>

typedef __attribute__((address_space(3))) void lds_void;

#define TTT_LDS_LOAD(op, soff) \
  "s_mov_b32 %0, m0\n\ts_mov_b32 m0, %1\n\ts_nop 0\n\t" op " %2, %3, " soff " offen lds\n\ts_mov_b32 m0, %0"

__device__ __forceinline__ uint32_t lds_base(void *lds) {
  return __builtin_amdgcn_readfirstlane((uint32_t)(uintptr_t)(lds_void *)lds);
}
__device__ __forceinline__ void dma16_untracked(__amdgpu_buffer_rsrc_t rs, void *lds, uint32_t voff) {
  uint32_t keep;
  asm volatile(TTT_LDS_LOAD("buffer_load_dwordx4", "0")
               : "=&s"(keep)
               : "s"(lds_base(lds)), "v"(voff), "s"(rs)
               : "memory");
}
__device__ __forceinline__ void dma16_untracked(__amdgpu_buffer_rsrc_t rs, void *lds, uint32_t voff, uint32_t soff) {
  uint32_t keep;
  asm volatile(TTT_LDS_LOAD("buffer_load_dwordx4", "%4")
               : "=&s"(keep)
               : "s"(lds_base(lds)), "v"(voff), "s"(rs), "s"(soff)
               : "memory");
}
__device__ __forceinline__ void dma4_untracked(__amdgpu_buffer_rsrc_t rs, void *lds, uint32_t voff, uint32_t soff) {
  uint32_t keep;
  asm volatile(TTT_LDS_LOAD("buffer_load_dword", "%4")
               : "=&s"(keep)
               : "s"(lds_base(lds)), "v"(voff), "s"(rs), "s"(soff)
               : "memory");
}

#undef TTT_LDS_LOAD
