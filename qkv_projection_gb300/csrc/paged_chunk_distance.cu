// Attention of many rows whose scores lose with distance.
#include "paged_chunk.cuh"

namespace kaio {

cudaError_t launch_paged_chunk_distance(FloatType t, const PagedParams& p, void* workspace, int num_sms,
                                        cudaStream_t stream) {
  return p.cap_in != 0.f ? launch_chunk<Form::kCappedDistance>(t, p, workspace, num_sms, stream, kOwnWaitLimit)
                         : launch_chunk<Form::kDistance>(t, p, workspace, num_sms, stream, kOwnWaitLimit);
}

unsigned read_and_clear_chunk_distance_errors() { return read_and_clear_errors(); }

}  // namespace kaio
