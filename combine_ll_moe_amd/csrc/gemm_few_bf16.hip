// Products grouped by expert, few rows: bf16 weights, and the choice by type.
#include "gemm_few.h"

namespace llmoe {

hipError_t launch_gemm_few(const GemmParams& p, int most, hipStream_t stream) {
  if (p.weight == kWeightFp8) return launch_gemm_few_fp8(p, most, stream);
  if (p.weight == kWeightInt4) return launch_gemm_few_int4(p, most, stream);
  return p.gated ? launch<kWeightBf16, 128, true, false>(p, most, stream)
                 : launch<kWeightBf16, 128, false, false>(p, most, stream);
}

}  // namespace llmoe
