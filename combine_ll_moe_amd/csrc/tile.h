// What the tiled products share: copies straight into LDS that stay under way
// across barriers, and the order in which the XCDs take tiles.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "expert_gemm.h"
#include "kernels.h"

namespace llmoe {

typedef __attribute__((address_space(3))) uint8_t LdsByte;
constexpr int kStep = 128;  // bytes of a row in a k step

// 16 bytes a lane (or 4) from a descriptor to LDS, lane after lane.
__device__ __forceinline__ void copy16(Rsrc from, uint8_t* lds, uint32_t off) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(from, (LdsByte*)lds, 16, (int)off, 0, 0, 0);
}
__device__ __forceinline__ void copy4(Rsrc from, uint8_t* lds, uint32_t off) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(from, (LdsByte*)lds, 4, (int)off, 0, 0, 0);
}

// s_waitcnt vmcnt(N) alone.
template <int N>
__device__ __forceinline__ void wait_loads() {
  static_assert(N < 64);
  __builtin_amdgcn_s_waitcnt(0x0F70 | (N & 15) | (N >> 4) << 14);
}

// A barrier alone: what is under way stays so.
__device__ __forceinline__ void meet() {
  __builtin_amdgcn_sched_barrier(0);
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

// Which tile workgroup b of `total` takes: the XCDs, to which workgroups are
// dealt in turn, take runs of the tiles, in which neighbours share operands.
__device__ __forceinline__ uint32_t run_of_xcd(uint32_t b, uint32_t total) {
  const uint32_t x = b % kXcds, whole = total / kXcds, more = total % kXcds;
  return x * whole + (x < more ? x : more) + b / kXcds;
}

}  // namespace llmoe
