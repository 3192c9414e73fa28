// Launcher of the root-mean-square norm.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace llmoe {

struct NormParams {
  const uint8_t* x;          // bf16 or fp32 [num_tokens, hidden]
  const uint8_t* residual;   // bf16, or null
  const uint8_t* weight;     // bf16 [hidden]
  uint8_t* residual_out;     // bf16, or null
  uint8_t* out;              // bf16 or e4m3
  float* out_scales;         // fp8: [num_tokens, hidden / 128]
  int num_tokens;
  int hidden;
  float eps;
  int x_fp32;
  int out_fp8;
};

constexpr int kNormMaxHidden = 32768;

hipError_t launch_norm(const NormParams& p, hipStream_t stream);

}  // namespace llmoe
