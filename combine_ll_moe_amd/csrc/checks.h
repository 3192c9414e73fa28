// Argument checks shared by the C ABI of the operators beside the dispatch
// and the combine.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "ll_moe.h"

namespace llmoe {

inline bool aligned(const void* p, uintptr_t a) { return ((uintptr_t)p & (a - 1)) == 0; }

inline bool overlaps(const void* a, uint64_t a_bytes, const void* b, uint64_t b_bytes) {
  const uintptr_t a0 = (uintptr_t)a, b0 = (uintptr_t)b;
  return a && b && a0 < b0 + b_bytes && b0 < a0 + a_bytes;
}

inline int from_hip(hipError_t e) { return e == hipSuccess ? LL_MOE_SUCCESS : LL_MOE_HIP_ERROR; }

struct Span {
  const void* p;
  uint64_t bytes;
};

// Whether any written span overlaps a read one or another written one.
template <int R, int W>
bool clash(const Span (&reads)[R], const Span (&writes)[W]) {
  for (int i = 0; i < W; ++i) {
    for (int j = 0; j < R; ++j)
      if (overlaps(writes[i].p, writes[i].bytes, reads[j].p, reads[j].bytes)) return true;
    for (int j = 0; j < i; ++j)
      if (overlaps(writes[i].p, writes[i].bytes, writes[j].p, writes[j].bytes)) return true;
  }
  return false;
}

}  // namespace llmoe
