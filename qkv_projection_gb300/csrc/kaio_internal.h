// Internal (non-exported) declarations shared by the translation units of
// libkaio_qkv: kernel parameter blocks, launch plans and launchers.
#pragma once

#include <cuda.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cstddef>
#include <cstdint>

namespace kaio {

// ---------------------------------------------------------------- decode path
struct DecodeParams {
  const __half* x;          // [M, K]
  const uint32_t* w[3];     // [K/8, N] each
  const __half* s[3];       // [K/128, N] each
  __half* out[3];           // [M, N] each
  int M, N, K;
  int groups_per_proj;      // ceil(N / 256)
  int nkb;                  // K / 64
  long long units;          // 3 * groups_per_proj * nkb
  int ctas;                 // grid size
  int xmax_kb;              // k-blocks of x staged in shared memory at once
  float* partials;          // [ctas][2][8][32][8*mt] split-K partial sums
  unsigned* counters;       // [3 * groups_per_proj], zero between launches
};

struct DecodePlan {
  int mt;                   // 1: M <= 8, 2: M <= 16
  int groups_per_proj;
  int nkb;
  long long units;
  int ctas;
  int xmax_kb;
  size_t smem;
  size_t partial_floats;
  int counters;
};

// Stream-K mma.sync decode kernel, run only by the allocation-free entry point.
DecodePlan plan_decode(int M, int N, int K, int num_sms);

// Allocation-free decode launch: split-K scratch in a fixed device array of
// kNoAllocScratchBytes (the first 64 KiB hold group counters). `prm` needs only
// the tensors and M, N, K; the plan and scratch pointers are filled in here.
constexpr size_t kNoAllocScratchBytes = 8u << 20;
int noalloc_max_counters();
cudaError_t launch_decode_noalloc(DecodeParams prm, int dev, int num_sms, cudaStream_t stream);

// tcgen05 decode (M <= 16): 128-column tiles over the three projections, split
// over K across a cluster of S CTAs.
struct TcDecodePlan {
  bool ok;
  int tiles;   // ceil(N / 128)
  int ng;      // K / 128
  int S;       // cluster size
};
TcDecodePlan plan_tc_decode(int M, int N, int K, int dev);
cudaError_t launch_tc_decode(const __half* x, const uint32_t* const w[3], const __half* const s[3],
                             __half* const out[3], int M, int N, int K, const TcDecodePlan& pl,
                             cudaStream_t stream);
// The INT4 decode kernel with every pipeline wait limited to wait_ns (a test
// of the bounded-wait timeout path; the regular launch uses 2 s).
cudaError_t launch_tc_decode_wait_limit(const __half* x, const uint32_t* const w[3], const __half* const s[3],
                                        __half* const out[3], int M, int N, int K, const TcDecodePlan& pl,
                                        unsigned long long wait_ns, cudaStream_t stream);
// The same kernel for INT8 weights u32[K/4, N] (byte i = K-row 4r+i) with
// one f32 scale per projection.
TcDecodePlan plan_tc_decode_int8(int M, int N, int K, int dev);
cudaError_t launch_tc_decode_int8(const __half* x, const uint32_t* const w[3], const float scale[3],
                                  __half* const out[3], int M, int N, int K, const TcDecodePlan& pl,
                                  cudaStream_t stream);
unsigned read_and_clear_tc_decode_errors();

// ------------------------------------------------- per-group dequantisation
enum class FloatType { F32, F64, F16, BF16 };
// dx[i, j] = dy[i, j] * scale[i, j / group] over [outer, axis], in type t.
cudaError_t launch_dequant_group_backward(FloatType t, const void* dy, const void* scale, void* dx,
                                          int outer, int axis, int group, int num_sms, cudaStream_t stream);
// out[i, j] = t(q[i, j]) * scale[i, j / group], q int8 (or uint8 if q_unsigned).
cudaError_t launch_dequant_group_forward(FloatType t, bool q_unsigned, const void* q, const void* scale,
                                         void* out, int outer, int axis, int group, int num_sms,
                                         cudaStream_t stream);

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
constexpr size_t kPagedCounterBytes = 4096;
size_t paged_decode_workspace_bytes(int num_sms);
cudaError_t launch_paged_decode(FloatType t, PagedParams p, void* workspace, int num_sms, cudaStream_t stream);
size_t paged_chunk_workspace_bytes(int num_sms);
cudaError_t launch_paged_chunk(FloatType t, const PagedParams& p, void* workspace, int num_sms, cudaStream_t stream);
unsigned read_and_clear_chunk_errors();

// ------------------------------------------------- tensor-core (tcgen05) paths
struct GemmShape {
  int M, N, K;              // C[M, N] = sum_k Aop[M, k] * Bop[k, N]
};

// Dense f16 x f16 -> f32 accumulate, stored as f32 or (c_f16) f16. a_mn / b_mn
// select the operand storage:
//   Aop K-major: A stored [M][K];  MN-major: A stored [K][M]
//   Bop K-major: B stored [N][K];  MN-major: B stored [K][N]
cudaError_t launch_tc_gemm(const void* a, const void* b, void* c, GemmShape sh, bool a_mn,
                           bool b_mn, bool c_f16, int num_sms, cudaStream_t stream);

// W4A16 fused projection for M >= 17 on tcgen05 (weights as the TMEM operand).
cudaError_t launch_tc_w4a16(const __half* x, const uint32_t* const w[3], const __half* const s[3],
                            __half* const out[3], int M, int N, int K, int num_sms,
                            cudaStream_t stream);
// W8A16 prefill: packed INT8 weights u32[K/4, N] (byte i = K-row 4r+i), one
// f32 scale per projection.
cudaError_t launch_tc_w8a16(const __half* x, const uint32_t* const w[3], const float scale[3],
                            __half* const out[3], int M, int N, int K, int num_sms,
                            cudaStream_t stream);

// Bit-exact dequantisation (debug / test entry).
cudaError_t launch_dequant_debug(const uint32_t* w, const __half* s, __half* out, int K, int N,
                                 int variant, cudaStream_t stream);

// Device error word (bounded-wait timeouts), read and cleared by the host API.
constexpr unsigned kDevErrTimeoutHost = 1u;   // same bit as kDevErrTimeout in kaio_device.cuh
unsigned read_and_clear_tc_errors();

// Raise a kernel's dynamic shared memory limit once per (kernel, device):
// later calls (including those made while a stream is being captured into a
// CUDA graph) only look the pair up.
cudaError_t ensure_smem_limit(const void* kernel, int bytes);

// Driver entry point for tensor-map encoding (resolved once through the runtime).
// encode_tensor_map: any rank, strides in bytes of dimensions 1 and up, nothing kept.
CUresult encode_tensor_map(CUtensorMap* map, CUtensorMapDataType dtype, uint32_t rank, const void* base,
                           const uint64_t* dims, const uint64_t* strides, const uint32_t* box,
                           CUtensorMapSwizzle swz);
CUresult encode_tensor_map_2d(CUtensorMap* map, CUtensorMapDataType dtype, const void* base,
                              uint64_t inner, uint64_t outer, uint64_t row_bytes,
                              uint32_t box_inner, uint32_t box_outer, CUtensorMapSwizzle swz);

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
