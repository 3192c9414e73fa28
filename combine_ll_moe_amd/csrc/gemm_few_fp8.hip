// Products grouped by expert, few rows: fp8 weights.
#include "gemm_few.h"

namespace llmoe {

hipError_t launch_gemm_few_fp8(const GemmParams& p, int most, hipStream_t stream) {
  if (p.out_fp8) return launch<kWeightFp8, 128, true, true>(p, most, stream);
  return p.gated ? launch<kWeightFp8, 128, true, false>(p, most, stream)
                 : launch<kWeightFp8, 128, false, false>(p, most, stream);
}

}  // namespace llmoe
