// Dense block-scaled fp8 products: what the kernels and the C ABI share.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace llmoe {

enum : int { kOutBf16 = 0, kOutFp8 = 1, kOutFp32 = 2 };

struct DenseParams {
  const uint8_t* a;        // e4m3 [m, k]
  const float* a_scales;   // [m, k / 128]
  const uint8_t* w;        // e4m3 [n or 2n, k]
  const float* w_scales;   // [ceil(rows / 128), k / 128]
  const float* addend;     // [m, n], or null
  uint8_t* out;            // [m, n]
  float* out_scales;       // fp8: [m, n / 128]
  float* partial;          // workspace: fp32 sums
  int m;
  int n;
  int k;
  int gated;               // W has n gate rows, then n up rows
  int out_type;
};

hipError_t launch_dense(const DenseParams& p, hipStream_t stream);

}  // namespace llmoe
