// Attention of few rows whose scores lose with distance.
#include "paged_decode.cuh"

namespace kaio {

cudaError_t launch_paged_decode_distance(FloatType t, const PagedParams& p, void* workspace, int num_sms,
                                         cudaStream_t stream) {
  return p.cap_in != 0.f ? launch_decode<Form::kCappedDistance>(t, p, workspace, num_sms, stream)
                         : launch_decode<Form::kDistance>(t, p, workspace, num_sms, stream);
}

}  // namespace kaio
