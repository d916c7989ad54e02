// Attention of many rows without a cap, slopes, prefixes or documents.
#include "paged_chunk.cuh"

namespace kaio {

size_t paged_chunk_workspace_bytes(int num_sms) {
  return kPagedCounterBytes + 32 + static_cast<size_t>(num_sms) * 2 * kRows * (128 + 1) * sizeof(float);
}

cudaError_t launch_paged_chunk(FloatType t, const PagedParams& p, void* workspace, int num_sms, cudaStream_t stream,
                               unsigned long long wait_ns) {
  return launch_chunk<Form::kPlain>(t, p, workspace, num_sms, stream, wait_ns);
}

unsigned read_and_clear_chunk_errors() { return read_and_clear_errors(); }

}  // namespace kaio
