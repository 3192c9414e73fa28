// Launcher of the routing: logits to picked experts and their weights.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace llmoe {

struct PickParams {
  const void* logits;        // fp32 or bf16 [num_tokens, num_experts]
  const float* bias;         // [num_experts], or null
  const int32_t* num_valid;  // rows that are routed, or null: all
  int32_t* topk_idx;         // [num_tokens, topk]
  float* topk_weights;       // [num_tokens, topk]
  int num_tokens;
  int num_experts;
  int topk;
  int num_groups;
  int topk_groups;
  int group_best;            // a group counts as the sum of its best 1 or 2
  int bf16;
  int sigmoid;               // else softmax
  int renormalize;
  float scale;
};

constexpr int kPickMaxExperts = 4096;
constexpr int kPickMaxGroups = 64;

hipError_t launch_pick(const PickParams& p, hipStream_t stream);

}  // namespace llmoe
