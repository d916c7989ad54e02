// Attention of many rows with a cap, prefixes or documents, but no slopes.
#include "paged_chunk.cuh"

namespace kaio {

cudaError_t launch_paged_chunk_scored(FloatType t, const PagedParams& p, void* workspace, int num_sms,
                                      cudaStream_t stream) {
  if (p.slopes) return launch_paged_chunk_distance(t, p, workspace, num_sms, stream);
  return p.cap_in != 0.f ? launch_chunk<Form::kCapped>(t, p, workspace, num_sms, stream, kOwnWaitLimit)
                         : launch_chunk<Form::kMasks>(t, p, workspace, num_sms, stream, kOwnWaitLimit);
}

unsigned read_and_clear_chunk_scored_errors() {
  const unsigned e = read_and_clear_errors(), d = read_and_clear_chunk_distance_errors();
  return e | d;
}

}  // namespace kaio
