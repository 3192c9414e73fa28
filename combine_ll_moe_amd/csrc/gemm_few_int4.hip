// Products grouped by expert, few rows: 4-bit weights.
#include "gemm_few.h"

namespace llmoe {
namespace {

template <int G>
hipError_t launch_group(const GemmParams& p, int most, hipStream_t stream) {
  return p.gated ? launch<kWeightInt4, G, true, false>(p, most, stream)
                 : launch<kWeightInt4, G, false, false>(p, most, stream);
}

}  // namespace

hipError_t launch_gemm_few_int4(const GemmParams& p, int most, hipStream_t stream) {
  return p.group == 128  ? launch_group<128>(p, most, stream)
         : p.group == 64 ? launch_group<64>(p, most, stream)
                         : launch_group<32>(p, most, stream);
}

}  // namespace llmoe
