// Host-side interface of the rotary and paged-attention kernels (rope.cu,
// paged_decode.cu, paged_chunk.cu), beside kaio_internal.h.
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

#include "../../include/kaio_qkv.h"
#include "kaio_internal.h"

namespace kaio {

// n / d for 0 <= n < 2^31 by one multiplication (round-up reciprocal).
struct FastDiv {
  uint32_t mul = 1, shift = 0, d = 1;
  FastDiv() = default;
  explicit FastDiv(uint32_t div) : d(div) {
    while ((1ull << shift) < div) ++shift;
    mul = static_cast<uint32_t>(((1ull << 32) * ((1ull << shift) - div)) / div + 1);
  }
#ifdef __CUDACC__
  __device__ __forceinline__ int div(int n) const {
    return static_cast<int>((__umulhi(static_cast<uint32_t>(n), mul) + static_cast<uint32_t>(n)) >> shift);
  }
#endif
};

// ----------------------------------------------- rotary positions, cache write
// Strides are in elements. kv_heads == 0: q alone (no cache).
struct RopeParams {
  const void *q, *k, *v;
  void *qo, *kc, *vc;
  long long q_ts, q_hs, qo_ts, qo_hs, k_ts, k_hs, v_ts, v_hs;   // token and head strides
  long long kc_ps, kc_ss, kc_hs, vc_ps, vc_ss, vc_hs;           // page, slot and head strides
  const int* slots;           // [tokens] page * page_size + slot; outside the cache: not stored
  const int* positions;       // [axes][tokens], axis stride pos_stride
  long long pos_stride;
  const float* inv_freq;      // [pairs]
  int tokens, q_heads, kv_heads, dim, pairs, axes;
  int section_end[4];         // first pair past each axis's section
  int num_pages, page_size;
  bool interleaved, inverse;
};
// A thread's units of work: up to two 16-byte vectors of one head (pairs that are whole
// vectors), or a head's row.
struct RopeUnits {
  bool vec;
  int rot, copy;                 // of a rotated and of a copied head
  explicit RopeUnits(const RopeParams& r)
      : vec(r.interleaved ? r.pairs % 4 == 0 : r.pairs % 8 == 0),
        rot(!vec ? 1 : r.interleaved ? (r.dim + 15) / 16 : r.pairs / 8 + (r.dim - 2 * r.pairs + 15) / 16),
        copy(!vec ? 1 : (r.dim + 15) / 16) {}
  // Of one token; the kernel counts them in 32 bits.
  int64_t per_token(const RopeParams& r) const {
    return (static_cast<int64_t>(r.q_heads) + r.kv_heads) * rot + static_cast<int64_t>(r.kv_heads) * copy;
  }
};
cudaError_t launch_rope(FloatType t, const RopeParams& r, int num_sms, cudaStream_t stream);

// ------------------------------------------------------------- paged attention
// Strides are in elements.
struct PagedParams {
  const void *q, *kc, *vc;
  void* out;
  float* lse;                 // [tokens][heads], natural logarithm; may be null
  long long q_ts, q_hs, o_ts, o_hs;
  long long k_ps, k_ss, k_hs, v_ps, v_ss, v_hs, table_stride;
  const int *table, *kv_lens, *q_starts;   // q_starts may be null: one token per sequence
  int batch, tokens, heads, kv_heads, group, dim;
  FastDiv group_div;          // group = heads / kv_heads
  int page_shift, num_pages, max_pages;
  bool causal;
  int window, sinks;          // window 0: none; both at most kPagedMaxLen
  float scale_log2;           // softmax scale * log2(e)
  float* part_o;              // [2 * ctas][rows][dim] partial outputs of split work
  float* part_l;              // [2 * ctas][rows] their log2-sum-exp2
  unsigned* counters;         // [ctas], zero between launches
};
constexpr int kPagedMaxLen = 1 << 30;
// Rows (tokens x query heads of one K/V head) that one CTA of the warp-MMA
// kernel takes at a time.
constexpr int kPagedDecodeRows = 16;
// Workspace layout: counters first, then the partial sums.
constexpr size_t kPagedCounterBytes = KAIO_PAGED_ATTENTION_COUNTERS;
size_t paged_decode_workspace_bytes(int num_sms);
cudaError_t launch_paged_decode(FloatType t, PagedParams p, void* workspace, int num_sms, cudaStream_t stream);
size_t paged_chunk_workspace_bytes(int num_sms);
// wait_ns: limit of the pipeline's waits, kOwnWaitLimit but in a test of the path that gives
// up, which is built for one type and width.
constexpr unsigned long long kOwnWaitLimit = ~0ull;
constexpr bool paged_chunk_limit_ok(FloatType t, int dim) { return t == FloatType::F16 && dim > 64; }
cudaError_t launch_paged_chunk(FloatType t, const PagedParams& p, void* workspace, int num_sms, cudaStream_t stream,
                               unsigned long long wait_ns);
unsigned read_and_clear_chunk_errors();

// A launch that may begin while the kernel before it in the stream still runs
// (programmatic dependent launch): the kernel waits for it (grid_dependency_wait)
// before it touches memory.
template <typename... Params, typename... Args>
cudaError_t launch_dependent(void (*kernel)(Params...), int grid, int threads, int smem, cudaStream_t stream,
                             const Args&... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(grid));
  cfg.blockDim = dim3(static_cast<unsigned>(threads));
  cfg.dynamicSmemBytes = static_cast<size_t>(smem);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

}  // namespace kaio
