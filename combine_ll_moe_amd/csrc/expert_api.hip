// C ABI of the operators around the expert side (declared in
// include/ll_moe.h): argument checks, then the launch on the caller's
// stream. Nothing here allocates, frees or synchronizes.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "expert_gemm.h"
#include "layout.h"
#include "ll_moe.h"
#include "norm.h"

using namespace llmoe;

namespace {

bool aligned(const void* p, uintptr_t a) { return ((uintptr_t)p & (a - 1)) == 0; }

bool overlaps(const void* a, uint64_t a_bytes, const void* b, uint64_t b_bytes) {
  const uintptr_t a0 = (uintptr_t)a, b0 = (uintptr_t)b;
  return a && b && a0 < b0 + b_bytes && b0 < a0 + a_bytes;
}

int from_hip(hipError_t e) { return e == hipSuccess ? LL_MOE_SUCCESS : LL_MOE_HIP_ERROR; }

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

bool gemm_sizes(int max_tokens, int n, int k, int num_experts, int act) {
  if (max_tokens < 1 || num_experts < 1 || num_experts > LL_MOE_SEND_MAX_EXPERTS) return false;
  if (n < 1 || n > LL_MOE_GEMM_MAX_COLUMNS || k < 1 || k > LL_MOE_GEMM_MAX_COLUMNS) return false;
  if ((int64_t)num_experts * max_tokens > INT32_MAX) return false;
  return act == LL_MOE_ACT_NONE || act == LL_MOE_ACT_SILU_MUL;
}

// One launch or two. The few kernel takes experts of up to kFewRows rows, the
// tile kernel those of more (64 experts of 4096 x 1536 bf16 weights, 100 rows
// each: 209 us in tiles against 297 in the few kernel, which reads the weights
// twice; the same for fp8, 390 against 476 with 7168 x 2048; 4-bit weights would be
// faster there, 217 against 276, and slower at uneven counts). Where no expert
// can have as many, one launch does. An empty second launch takes 4 us: calls
// that are short themselves, with at most 128 rows an expert and less than 256
// MiB of weights, do without it and leave every row to the few kernel (8
// experts of 1024 x 1024: 9.4 us against 13).
constexpr uint64_t kTileWeights = 256ull << 20;

int launch_gemm(const GemmParams& p, hipStream_t stream) {
  const uint64_t weights = (uint64_t)p.num_experts * (p.gated ? 2 : 1) * p.n * p.k;
  const uint64_t bytes = p.weight == kWeightBf16 ? 2 * weights : p.weight == kWeightFp8 ? weights : weights / 2;
  if (p.max_tokens <= kFewRows || (p.max_tokens <= 2 * kFewRows && bytes < kTileWeights))
    return from_hip(launch_gemm_few(p, INT32_MAX, stream));
  const hipError_t e = launch_gemm_few(p, kFewRows, stream);
  return from_hip(e != hipSuccess ? e : launch_gemm_tile(p, kFewRows, stream));
}

}  // namespace

extern "C" int ll_moe_expert_gemm(int max_tokens, int n, int k, int num_experts, int dtype, int act,
                                  int out_dtype, const void* a, const float* a_scales,
                                  const void* w, const float* w_scales, const int32_t* counts,
                                  void* out, float* out_scales, hipStream_t stream) {
  if (!gemm_sizes(max_tokens, n, k, num_experts, act)) return LL_MOE_INVALID_ARGUMENT;
  const bool fp8 = dtype == LL_MOE_FP8_E4M3, gated = act == LL_MOE_ACT_SILU_MUL;
  const bool out_fp8 = out_dtype == LL_MOE_FP8_E4M3;
  if (!fp8 && dtype != LL_MOE_BF16) return LL_MOE_INVALID_ARGUMENT;
  if (!out_fp8 && out_dtype != LL_MOE_BF16) return LL_MOE_INVALID_ARGUMENT;
  if (fp8 ? (k % kFp8Block || n % 16) : (k % 8 || n % 8)) return LL_MOE_INVALID_ARGUMENT;
  if (out_fp8 && (!fp8 || !gated || n % kFp8Block)) return LL_MOE_INVALID_ARGUMENT;
  if (!a || !w || !counts || !out || (fp8 && (!a_scales || !w_scales)) || (out_fp8 && !out_scales))
    return LL_MOE_INVALID_ARGUMENT;
  if (!aligned(a, 16) || !aligned(w, 16) || !aligned(out, 16) || !aligned(counts, 4) ||
      (fp8 && (!aligned(a_scales, 4) || !aligned(w_scales, 4))) ||
      (out_fp8 && !aligned(out_scales, 4)))
    return LL_MOE_INVALID_ARGUMENT;
  const uint64_t rows = (uint64_t)num_experts * max_tokens, rows_w = gated ? 2 * (uint64_t)n : n;
  const uint64_t kb = (uint64_t)k / kFp8Block, item = fp8 ? 1 : 2;
  const Span reads[] = {{a, rows * k * item},
                        {w, num_experts * rows_w * k * item},
                        {fp8 ? a_scales : nullptr, rows * kb * 4},
                        {fp8 ? w_scales : nullptr, num_experts * ((rows_w + 127) / 128) * kb * 4},
                        {counts, (uint64_t)num_experts * 4}};
  const Span writes[] = {{out, rows * n * (out_fp8 ? 1 : 2)},
                         {out_fp8 ? out_scales : nullptr, rows * (n / kFp8Block) * 4}};
  if (clash(reads, writes)) return LL_MOE_INVALID_ARGUMENT;

  GemmParams p = {};
  p.a = static_cast<const uint8_t*>(a);
  p.a_scales = a_scales;
  p.w = static_cast<const uint8_t*>(w);
  p.w_scales = w_scales;
  p.counts = counts;
  p.out = static_cast<uint8_t*>(out);
  p.out_scales = out_scales;
  p.max_tokens = max_tokens;
  p.num_experts = num_experts;
  p.n = n;
  p.k = k;
  p.weight = fp8 ? kWeightFp8 : kWeightBf16;
  p.gated = gated;
  p.out_fp8 = out_fp8;
  return launch_gemm(p, stream);
}

extern "C" int ll_moe_expert_gemm_w4(int max_tokens, int n, int k, int num_experts, int group,
                                     int act, const void* a, const void* w, const void* w_scales,
                                     const uint8_t* w_zeros, const int32_t* counts, void* out,
                                     hipStream_t stream) {
  if (!gemm_sizes(max_tokens, n, k, num_experts, act)) return LL_MOE_INVALID_ARGUMENT;
  if (group != 32 && group != 64 && group != 128) return LL_MOE_INVALID_ARGUMENT;
  if (k % group || n % 8) return LL_MOE_INVALID_ARGUMENT;
  if (!a || !w || !w_scales || !counts || !out) return LL_MOE_INVALID_ARGUMENT;
  if (!aligned(a, 16) || !aligned(w, 16) || !aligned(out, 16) || !aligned(counts, 4) ||
      !aligned(w_scales, 16) || !aligned(w_zeros, 8))
    return LL_MOE_INVALID_ARGUMENT;
  const bool gated = act == LL_MOE_ACT_SILU_MUL;
  const uint64_t rows = (uint64_t)num_experts * max_tokens, rows_w = gated ? 2 * (uint64_t)n : n;
  const uint64_t groups = num_experts * rows_w * (k / group);
  if (rows_w * (k / group) >= 1ull << 30) return LL_MOE_INVALID_ARGUMENT;  // 32-bit offsets of the scales
  const Span reads[] = {{a, rows * k * 2},
                        {w, num_experts * rows_w * k / 2},
                        {w_scales, groups * 2},
                        {w_zeros, groups},
                        {counts, (uint64_t)num_experts * 4}};
  const Span writes[] = {{out, rows * n * 2}};
  if (clash(reads, writes)) return LL_MOE_INVALID_ARGUMENT;

  GemmParams p = {};
  p.a = static_cast<const uint8_t*>(a);
  p.w = static_cast<const uint8_t*>(w);
  p.w_scales = w_scales;
  p.w_zeros = w_zeros;
  p.counts = counts;
  p.out = static_cast<uint8_t*>(out);
  p.max_tokens = max_tokens;
  p.num_experts = num_experts;
  p.n = n;
  p.k = k;
  p.group = group;
  p.weight = kWeightInt4;
  p.gated = gated;
  return launch_gemm(p, stream);
}

extern "C" int ll_moe_rms_norm(int num_tokens, int hidden, int x_dtype, int out_dtype, float eps,
                               const void* x, const void* residual, const void* weight,
                               void* residual_out, void* out, float* out_scales,
                               hipStream_t stream) {
  if (num_tokens < 0 || hidden < 1 || hidden > kNormMaxHidden || hidden % 8)
    return LL_MOE_INVALID_ARGUMENT;
  if (x_dtype != LL_MOE_BF16 && x_dtype != LL_MOE_FP32) return LL_MOE_INVALID_ARGUMENT;
  if (out_dtype != LL_MOE_BF16 && out_dtype != LL_MOE_FP8_E4M3) return LL_MOE_INVALID_ARGUMENT;
  const bool fp8 = out_dtype == LL_MOE_FP8_E4M3, wide = x_dtype == LL_MOE_FP32;
  if (fp8 && hidden % kFp8Block) return LL_MOE_INVALID_ARGUMENT;
  if (!(eps >= 0.0f) || eps > 3.4e38f) return LL_MOE_INVALID_ARGUMENT;
  if (num_tokens > 0) {
    if (!x || !weight || !out || (fp8 && !out_scales)) return LL_MOE_INVALID_ARGUMENT;
    if (!aligned(x, 16) || !aligned(weight, 16) || !aligned(out, 16) || !aligned(residual, 16) ||
        !aligned(residual_out, 16) || (fp8 && !aligned(out_scales, 4)))
      return LL_MOE_INVALID_ARGUMENT;
    const uint64_t values = (uint64_t)num_tokens * hidden;
    // residual_out may be residual itself (each row is read before it is
    // written, by the workgroup that writes it); nothing else may overlap
    const Span reads[] = {{x, values * (wide ? 4 : 2)},
                          {weight, (uint64_t)hidden * 2},
                          {residual_out == residual ? nullptr : residual, values * 2}};
    const Span writes[] = {{residual_out, values * 2},
                           {out, values * (fp8 ? 1 : 2)},
                           {fp8 ? out_scales : nullptr, values / kFp8Block * 4}};
    if (clash(reads, writes)) return LL_MOE_INVALID_ARGUMENT;
  }
  NormParams p;
  p.x = static_cast<const uint8_t*>(x);
  p.residual = static_cast<const uint8_t*>(residual);
  p.weight = static_cast<const uint8_t*>(weight);
  p.residual_out = static_cast<uint8_t*>(residual_out);
  p.out = static_cast<uint8_t*>(out);
  p.out_scales = out_scales;
  p.num_tokens = num_tokens;
  p.hidden = hidden;
  p.eps = eps;
  p.x_fp32 = wide;
  p.out_fp8 = fp8;
  return from_hip(launch_norm(p, stream));
}
