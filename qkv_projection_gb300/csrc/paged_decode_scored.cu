// Attention of few rows whose scores are capped or lose with distance, or whose keys are
// limited by prefixes and documents.
#include "paged_decode.cuh"

namespace kaio {

cudaError_t launch_paged_decode_scored(FloatType t, const PagedParams& p, void* workspace, int num_sms,
                                       cudaStream_t stream) {
  return launch_decode<true>(t, p, workspace, num_sms, stream);
}

}  // namespace kaio
