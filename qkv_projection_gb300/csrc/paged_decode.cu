// Attention of few rows without a cap, slopes, prefixes or documents.
#include "paged_decode.cuh"

namespace kaio {

size_t paged_decode_workspace_bytes(int num_sms) {
  const size_t ctas = static_cast<size_t>(num_sms) * kCtasPerSm;
  return kPagedCounterBytes + 2 * ctas * kRows * (128 + 1) * sizeof(float);
}

cudaError_t launch_paged_decode(FloatType t, const PagedParams& p, void* workspace, int num_sms, cudaStream_t stream) {
  return launch_decode<Form::kPlain>(t, p, workspace, num_sms, stream);
}

}  // namespace kaio
