// Filling LDS straight from memory, with no register between: for the kernels of
// attention and the gated feed-forward product.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace dmuon {

// Byte address of a __shared__ location in the LDS aperture.
typedef __attribute__((address_space(3))) char* lds_ptr_t;
__device__ __forceinline__ uint32_t lds_address(lds_ptr_t p) { return static_cast<uint32_t>(reinterpret_cast<size_t>(p)); }
__device__ __forceinline__ uint32_t lds_address(const char* p) { return lds_address((lds_ptr_t)p); }   // address-space cast

// A workgroup-uniform pointer moved into SGPRs (it is computed from the block
// index and arguments, but not always provably uniform to the compiler).
__device__ __forceinline__ const char* uniform_ptr(const void* p) {
  const uint64_t v = reinterpret_cast<uint64_t>(p);
  const uint32_t lo = __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(v));
  const uint32_t hi = __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(v >> 32));
  return reinterpret_cast<const char*>((static_cast<uint64_t>(hi) << 32) | lo);
}

// global_load_lds_dwordx4: 16 bytes from base + voff (per lane) to
// LDS[lds_dst + 16 * lane].  Issued through asm so the compiler's wait-count
// pass does not treat it as an LDS operation of unknown completion order
// (which would force a full LDS wait before every fragment use); callers wait
// with an explicit vmcnt(0) and a barrier before reading the data.  M0 is set
// here and used by nothing else in the kernels that call this; s_nop covers the
// M0 hazard.
__device__ __forceinline__ void lds_dma16(const void* base, uint32_t voff, uint32_t lds_dst) {
  asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, %1" ::"v"(voff), "s"(base),
               "s"(lds_dst)
               : "memory");
}

// The same of 4 bytes a lane, to LDS[lds_dst + 4 * lane].
__device__ __forceinline__ void lds_dma4(const void* base, uint32_t voff, uint32_t lds_dst) {
  asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tglobal_load_lds_dword %0, %1" ::"v"(voff), "s"(base), "s"(lds_dst) : "memory");
}

}  // namespace dmuon
