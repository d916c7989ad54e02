// Attention of few rows with a cap, prefixes or documents, but no slopes.
#include "paged_decode.cuh"

namespace kaio {

cudaError_t launch_paged_decode_scored(FloatType t, const PagedParams& p, void* workspace, int num_sms,
                                       cudaStream_t stream) {
  if (p.slopes) return launch_paged_decode_distance(t, p, workspace, num_sms, stream);
  return p.cap_in != 0.f ? launch_decode<Form::kCapped>(t, p, workspace, num_sms, stream)
                         : launch_decode<Form::kMasks>(t, p, workspace, num_sms, stream);
}

}  // namespace kaio
