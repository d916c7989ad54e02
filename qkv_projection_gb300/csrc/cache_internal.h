// Host-side interface of the paged cache's upkeep (cache.cu).
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

#include "attention_internal.h"

namespace kaio {

// What one launch takes: caches in its parameters, rows and pages in shared memory (3 words
// a row, a bit a page).
constexpr int kCacheMaxCaches = 64;
constexpr int kCacheMaxBatch = 8192;
constexpr int kCacheMaxPages = 1 << 23;
constexpr int kCacheSmem = 192 * 1024;

// Strides and sizes in pieces of 16 bytes.
struct CacheCopyParams {
  // A page: `inner` consecutive pieces, `middle` times, and so on outwards.
  struct Cache {
    void* base;
    long long page_stride, middle_stride, outer_stride;
    int inner, middle;
  } cache[kCacheMaxCaches];
  const int *src, *dst;
  int num_pages, pieces, blocks;      // pieces of a page; CTAs that copy it
};
int cache_copy_blocks(int pieces);
// dense: every page is one run of pieces.
cudaError_t launch_cache_copy(const CacheCopyParams& p, int caches, int pairs, bool dense, cudaStream_t stream);

struct CacheParams {
  int *page_refs, *page_table, *kv_lens;
  const int *parents, *q_starts, *new_lens;
  int *slots, *src, *dst;
  long long table_stride;
  int batch, max_pages, num_pages, page_size;
  int tokens, max_moves;
  FastDiv page_div;
  int most_ctas;        // limit of a cluster; 0: the device's
  int warp_words;       // set by the launch: words of 32 pages that a warp looks after
};
// cudaErrorNotSupported: the pool's words do not fit in the shared memory of as many CTAs as can be placed.
cudaError_t launch_cache_fork(const CacheParams& p, cudaStream_t stream);
cudaError_t launch_cache_append(const CacheParams& p, cudaStream_t stream);
cudaError_t launch_cache_truncate(const CacheParams& p, cudaStream_t stream);
cudaError_t launch_cache_compact(const CacheParams& p, cudaStream_t stream);

}  // namespace kaio
