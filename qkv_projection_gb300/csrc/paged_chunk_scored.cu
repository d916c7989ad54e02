// Attention of many rows whose scores are capped or lose with distance, or whose keys are
// limited by prefixes and documents.
#include "paged_chunk.cuh"

namespace kaio {

cudaError_t launch_paged_chunk_scored(FloatType t, const PagedParams& p, void* workspace, int num_sms,
                                      cudaStream_t stream) {
  return launch_chunk<true>(t, p, workspace, num_sms, stream, kOwnWaitLimit);
}

unsigned read_and_clear_chunk_scored_errors() { return read_and_clear_errors(); }

}  // namespace kaio
