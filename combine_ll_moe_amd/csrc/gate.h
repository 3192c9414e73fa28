// Launcher of the router's logits.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace llmoe {

struct GateParams {
  const uint8_t* x;     // bf16 [num_tokens, hidden]
  const uint8_t* w;     // bf16 or fp32 [num_experts, hidden]
  float* logits;        // [num_tokens, num_experts]
  int num_tokens;
  int hidden;
  int num_experts;
  int w_fp32;
};

constexpr int kGateMaxHidden = 32768;
constexpr int kGateMaxExperts = 4096;

hipError_t launch_gate(const GateParams& p, hipStream_t stream);

}  // namespace llmoe
