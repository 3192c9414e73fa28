// C ABI of the router and the dense products (declared in include/ll_moe.h):
// argument checks, then the launch on the caller's stream. Nothing here
// allocates, frees or synchronizes.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <cmath>

#include "checks.h"
#include "dense.h"
#include "gate.h"
#include "layout.h"
#include "ll_moe.h"
#include "pick.h"

using namespace llmoe;

extern "C" int ll_moe_gate(int num_tokens, int hidden, int num_experts, int weight_dtype, const void* x,
                           const void* weight, float* logits, hipStream_t stream) {
  if (num_tokens < 0 || hidden < 1 || hidden > kGateMaxHidden || hidden % 8) return LL_MOE_INVALID_ARGUMENT;
  if (num_experts < 1 || num_experts > kGateMaxExperts) return LL_MOE_INVALID_ARGUMENT;
  if (weight_dtype != LL_MOE_BF16 && weight_dtype != LL_MOE_FP32) return LL_MOE_INVALID_ARGUMENT;
  const bool wide = weight_dtype == LL_MOE_FP32;
  if (num_tokens > 0) {
    if (!x || !weight || !logits) return LL_MOE_INVALID_ARGUMENT;
    if (!aligned(x, 16) || !aligned(weight, 16) || !aligned(logits, 16)) return LL_MOE_INVALID_ARGUMENT;
    const Span reads[] = {{x, (uint64_t)num_tokens * hidden * 2},
                          {weight, (uint64_t)num_experts * hidden * (wide ? 4 : 2)}};
    const Span writes[] = {{logits, (uint64_t)num_tokens * num_experts * 4}};
    if (clash(reads, writes)) return LL_MOE_INVALID_ARGUMENT;
  }
  GateParams p;
  p.x = static_cast<const uint8_t*>(x);
  p.w = static_cast<const uint8_t*>(weight);
  p.logits = logits;
  p.num_tokens = num_tokens;
  p.hidden = hidden;
  p.num_experts = num_experts;
  p.w_fp32 = wide;
  return from_hip(launch_gate(p, stream));
}

extern "C" int ll_moe_route(int num_tokens, int num_experts, int topk, int logits_dtype, int score, int num_groups,
                            int topk_groups, int group_best, int renormalize, float scale, const void* logits,
                            const float* bias, const int32_t* num_valid, int32_t* topk_idx, float* topk_weights,
                            hipStream_t stream) {
  if (num_tokens < 0 || num_experts < 1 || num_experts > kPickMaxExperts) return LL_MOE_INVALID_ARGUMENT;
  if (logits_dtype != LL_MOE_BF16 && logits_dtype != LL_MOE_FP32) return LL_MOE_INVALID_ARGUMENT;
  if (score != LL_MOE_SCORE_SOFTMAX && score != LL_MOE_SCORE_SIGMOID) return LL_MOE_INVALID_ARGUMENT;
  if (num_groups < 1 || num_groups > kPickMaxGroups || num_experts % num_groups) return LL_MOE_INVALID_ARGUMENT;
  const int per = num_experts / num_groups;
  if (topk_groups < 1 || topk_groups > num_groups) return LL_MOE_INVALID_ARGUMENT;
  if ((group_best != 1 && group_best != 2) || (num_groups > 1 && group_best > per)) return LL_MOE_INVALID_ARGUMENT;
  if (topk < 1 || topk > LL_MOE_MAX_TOPK || topk > topk_groups * per) return LL_MOE_INVALID_ARGUMENT;
  if (renormalize != 0 && renormalize != 1) return LL_MOE_INVALID_ARGUMENT;
  if (!std::isfinite(scale)) return LL_MOE_INVALID_ARGUMENT;
  if ((int64_t)num_tokens * topk > INT32_MAX) return LL_MOE_INVALID_ARGUMENT;
  if (num_tokens > 0) {
    if (!logits || !topk_idx || !topk_weights) return LL_MOE_INVALID_ARGUMENT;
    if (!aligned(logits, 16) || !aligned(bias, 4) || !aligned(num_valid, 4) || !aligned(topk_idx, 4) ||
        !aligned(topk_weights, 4))
      return LL_MOE_INVALID_ARGUMENT;
    const uint64_t picks = (uint64_t)num_tokens * topk;
    const Span reads[] = {{logits, (uint64_t)num_tokens * num_experts * (logits_dtype == LL_MOE_FP32 ? 4 : 2)},
                          {bias, (uint64_t)num_experts * 4},
                          {num_valid, 4}};
    const Span writes[] = {{topk_idx, picks * 4}, {topk_weights, picks * 4}};
    if (clash(reads, writes)) return LL_MOE_INVALID_ARGUMENT;
  }
  PickParams p;
  p.logits = logits;
  p.bias = bias;
  p.num_valid = num_valid;
  p.topk_idx = topk_idx;
  p.topk_weights = topk_weights;
  p.num_tokens = num_tokens;
  p.num_experts = num_experts;
  p.topk = topk;
  p.num_groups = num_groups;
  p.topk_groups = topk_groups;
  p.group_best = group_best;
  p.bf16 = logits_dtype == LL_MOE_BF16;
  p.sigmoid = score == LL_MOE_SCORE_SIGMOID;
  p.renormalize = renormalize;
  p.scale = scale;
  return from_hip(launch_pick(p, stream));
}

extern "C" int ll_moe_dense_gemm(int num_tokens, int n, int k, int act, int out_dtype, const void* a,
                                 const float* a_scales, const void* w, const float* w_scales, const float* addend,
                                 void* out, float* out_scales, void* workspace, hipStream_t stream) {
  if (num_tokens < 0 || n < 1 || n > LL_MOE_GEMM_MAX_COLUMNS || n % 16) return LL_MOE_INVALID_ARGUMENT;
  if (k < 1 || k > LL_MOE_GEMM_MAX_COLUMNS || k % kFp8Block) return LL_MOE_INVALID_ARGUMENT;
  if (act != LL_MOE_ACT_NONE && act != LL_MOE_ACT_SILU_MUL) return LL_MOE_INVALID_ARGUMENT;
  const bool gated = act == LL_MOE_ACT_SILU_MUL, fp8 = out_dtype == LL_MOE_FP8_E4M3, wide = out_dtype == LL_MOE_FP32;
  if (!fp8 && !wide && out_dtype != LL_MOE_BF16) return LL_MOE_INVALID_ARGUMENT;
  if (gated ? wide || addend : fp8) return LL_MOE_INVALID_ARGUMENT;
  if (fp8 && n % kFp8Block) return LL_MOE_INVALID_ARGUMENT;
  if (num_tokens > 0) {
    if (!a || !a_scales || !w || !w_scales || !out || !workspace || (fp8 && !out_scales))
      return LL_MOE_INVALID_ARGUMENT;
    if (!aligned(a, 16) || !aligned(w, 16) || !aligned(out, 16) || !aligned(addend, 16) || !aligned(workspace, 16) ||
        !aligned(a_scales, 4) || !aligned(w_scales, 4) || (fp8 && !aligned(out_scales, 4)))
      return LL_MOE_INVALID_ARGUMENT;
    const uint64_t rows = num_tokens, rows_w = gated ? 2 * (uint64_t)n : n, kb = (uint64_t)k / kFp8Block;
    // out may be the addend itself (each value is read before it is written,
    // by the thread that writes it); nothing else may overlap
    const Span reads[] = {{a, rows * k},
                          {a_scales, rows * kb * 4},
                          {w, rows_w * k},
                          {w_scales, (rows_w + 127) / 128 * kb * 4},
                          {wide && addend == out ? nullptr : addend, rows * n * 4}};
    const Span writes[] = {{out, rows * n * (fp8 ? 1 : wide ? 4 : 2)},
                           {fp8 ? out_scales : nullptr, rows * (n / kFp8Block) * 4},
                           {workspace, LL_MOE_DENSE_WORKSPACE}};
    if (clash(reads, writes)) return LL_MOE_INVALID_ARGUMENT;
  }
  DenseParams p;
  p.a = static_cast<const uint8_t*>(a);
  p.a_scales = a_scales;
  p.w = static_cast<const uint8_t*>(w);
  p.w_scales = w_scales;
  p.addend = addend;
  p.out = static_cast<uint8_t*>(out);
  p.out_scales = out_scales;
  p.partial = static_cast<float*>(workspace);
  p.m = num_tokens;
  p.n = n;
  p.k = k;
  p.gated = gated;
  p.out_type = fp8 ? kOutFp8 : wide ? kOutFp32 : kOutBf16;
  return from_hip(launch_dense(p, stream));
}
