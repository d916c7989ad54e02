// Upkeep of a paged cache: copies of pages, and the bookkeeping of which sequence holds
// which (forks, appended and dropped positions, compaction).
//
// The books are three arrays: page_refs[p] (how many places of the table hold page p; 0:
// free), page_table[b][i] and kv_lens[b]. Row b holds its first ceil(kv_lens[b] / page_size)
// places. All results are integers that follow from the books alone, whatever the order in
// which the GPU gets to them.
//
// What bounds the bookkeeping is latency: a step looks at some hundred rows and, to find free
// pages, at page_refs once (2 MB for half a million pages: 0.3 us). So each operator is one launch
// (the fork of a large table two), and where all pages have to be counted before any can be given
// out, the kernel is one CTA, or one cluster of up to 16, whose CTAs can wait for one another without a workspace.
// Of the GPU's time (in a graph) a step of 62 sequences takes 7.5 us (pages and slots 5, the cut 2.5), 256
// sequences with 52000 new positions in a pool of 250000 pages 15, a compaction of half a million pages 14-17
// (4700 cycles to count, 5000 for the table, 1000-2500 each time the cluster meets), a fork of 64 rows 2.9, of 512 rows
// with 960000 places 6.6. Among others, not in a graph, a call is bound by the host: 2.3 us for a cut, 4.5 where
// results are made.
#include <algorithm>
#include <cstdint>

#include "cache_internal.h"
#include "kaio_device.cuh"

namespace kaio {
namespace {

// ------------------------------------------------------------------- copying
// Page src[i] to page dst[i] of every cache: blocks of kCopyThreads x kCopyVecs 16-byte pieces, four
// loads of a thread in flight. Bound by memory: 500 pages of 64 KB in 16 caches, 1.05 GB, take 155.6 us, 6.74
// TB/s, what a plain copy reaches; 4 pages in 64 caches 3.1 us of the GPU and 6.4 of the host, which
// looks at 64 tensors.
constexpr int kCopyThreads = 256, kCopyVecs = 4;

template <bool kDense>
__global__ void __launch_bounds__(kCopyThreads) cache_copy_kernel(const __grid_constant__ CacheCopyParams p) {
  allow_dependents_launch();
  grid_dependency_wait();
  const int pair = blockIdx.x / p.blocks, block = blockIdx.x - pair * p.blocks;
  const int from = p.src[pair], to = p.dst[pair];
  if (from < 0 || from >= p.num_pages || to < 0 || to >= p.num_pages || from == to) return;
  const CacheCopyParams::Cache& c = p.cache[blockIdx.y];
  const uint4* src = static_cast<const uint4*>(c.base) + from * c.page_stride;
  uint4* dst = static_cast<uint4*>(c.base) + to * c.page_stride;
  uint4 v[kCopyVecs];
  long long at[kCopyVecs];
#pragma unroll
  for (int k = 0; k < kCopyVecs; ++k) {
    const int i = (block * kCopyVecs + k) * kCopyThreads + threadIdx.x;
    at[k] = -1;
    if (i < p.pieces) {
      if (kDense) {
        at[k] = i;
      } else {
        const int row = i / c.inner, outer = row / c.middle;
        at[k] = i - row * c.inner + (row - outer * c.middle) * c.middle_stride + outer * c.outer_stride;
      }
      v[k] = src[at[k]];
    }
  }
#pragma unroll
  for (int k = 0; k < kCopyVecs; ++k)
    if (at[k] >= 0) dst[at[k]] = v[k];
}

// --------------------------------------------------------------- bookkeeping
// Places that a row of this length holds.
__device__ __forceinline__ int places(const CacheParams& p, int len) {
  len = max(len, 0);
  const int whole = p.page_div.div(len);
  return min(whole + (whole * p.page_size < len), p.max_pages);
}
__device__ __forceinline__ bool is_page(const CacheParams& p, int id) { return id >= 0 && id < p.num_pages; }

// All threads of the cluster meet; what each wrote, the others see.
__device__ __forceinline__ void cluster_meet() {
  __syncwarp();
  cluster_sync_all();
}

// Row b becomes a copy of row parents[b], all at once: a CTA takes a few columns of all rows,
// whose entries it reads before it writes any. References change only where a place does, so
// what parent and row share already costs nothing. Lengths may be written once every CTA has
// read them: by the kernel itself where its CTAs are one cluster (kOne), by another one otherwise.
constexpr int kForkThreads = 512;
constexpr int kNotHeld = INT32_MIN;                          // (what stands in a held place may be that, too: no page)

template <bool kOne>
__global__ void __launch_bounds__(kForkThreads) cache_fork_kernel(const __grid_constant__ CacheParams p, int cols_log2) {
  extern __shared__ int smem[];
  int* lens = smem;                                          // [batch]
  int* parents = lens + p.batch;                             // [batch] -1: the row stays
  int* tile = parents + p.batch;                             // [batch][cols]
  const int cols = 1 << cols_log2, col0 = blockIdx.x * cols, n = p.batch * cols;
  allow_dependents_launch();
  grid_dependency_wait();
  for (int row = threadIdx.x; row < p.batch; row += kForkThreads) {
    const int parent = p.parents[row];
    lens[row] = p.kv_lens[row];
    parents[row] = parent < 0 || parent >= p.batch ? -1 : parent;
  }
  __syncthreads();
#pragma unroll 4
  for (int i = threadIdx.x; i < n; i += kForkThreads) {
    const int row = i >> cols_log2, col = col0 + (i & (cols - 1));
    tile[i] = col < places(p, lens[row]) ? p.page_table[row * p.table_stride + col] : kNotHeld;
  }
  if (kOne) cluster_meet();
  else __syncthreads();
#pragma unroll 4
  for (int i = threadIdx.x; i < n; i += kForkThreads) {
    const int row = i >> cols_log2, c = i & (cols - 1), parent = parents[row];
    if (parent < 0) continue;
    const int before = tile[i], now = tile[(parent << cols_log2) + c];
    if (before == now && now != kNotHeld) continue;
    if (is_page(p, before)) atomicSub(p.page_refs + before, 1);
    if (now != kNotHeld || col0 + c < places(p, lens[parent])) p.page_table[row * p.table_stride + col0 + c] = now;
    if (is_page(p, now)) atomicAdd(p.page_refs + now, 1);
  }
  if (kOne && blockIdx.x == 0) {
    for (int row = threadIdx.x; row < p.batch; row += kForkThreads)
      if (parents[row] >= 0) p.kv_lens[row] = lens[parents[row]];
  }
}

// The lengths of the fork, once all places have been read by them.
constexpr int kLensThreads = 1024;
__global__ void __launch_bounds__(kLensThreads) cache_fork_lens_kernel(const __grid_constant__ CacheParams p) {
  allow_dependents_launch();
  grid_dependency_wait();
  constexpr int kMine = kCacheMaxBatch / kLensThreads;
  int len[kMine];
#pragma unroll
  for (int k = 0; k < kMine; ++k) {
    const int row = threadIdx.x + k * kLensThreads;
    if (row < p.batch) {
      const int parent = p.parents[row];
      len[k] = p.kv_lens[parent < 0 || parent >= p.batch ? row : parent];
    }
  }
  __syncthreads();
#pragma unroll
  for (int k = 0; k < kMine; ++k) {
    const int row = threadIdx.x + k * kLensThreads;
    if (row < p.batch) p.kv_lens[row] = len[k];
  }
}

// A row is cut to new_lens[b] where that is less: a CTA for each row.
constexpr int kCutThreads = 128;
__global__ void __launch_bounds__(kCutThreads) cache_truncate_kernel(const __grid_constant__ CacheParams p) {
  allow_dependents_launch();
  grid_dependency_wait();
  const int row = blockIdx.x, len = p.kv_lens[row], kept = max(p.new_lens[row], 0);
  if (kept >= len) return;
  const int end = places(p, len);
  for (int i = places(p, kept) + threadIdx.x; i < end; i += kCutThreads) {
    const int id = p.page_table[row * p.table_stride + i];
    if (is_page(p, id)) atomicSub(p.page_refs + id, 1);
  }
  __syncthreads();                                           // all have read the length
  if (threadIdx.x == 0) p.kv_lens[row] = kept;
}

// ------------------------------------------- one cluster over the whole pool
constexpr int kMaxCtas = 16, kThreads = 1024, kWarps = kThreads / 32;
__device__ __forceinline__ int cluster_ctas() { return static_cast<int>(gridDim.x); }

// Pages [first, first + 32 words) belong to one warp; which of them are free is kept in shared
// memory, a bit each, and `before` becomes how many free ones lie before the warp's.
struct Pool {
  int words;            // of 32 pages
  int first;
  uint32_t* mask;       // this warp's
  int before, free;     // before this warp's pages; in the whole pool
};

struct PoolShared {
  int warp_free[kWarps], cta_free;
  int below;            // compaction: free pages below the line
};

__device__ __forceinline__ int remote(const int* p, int cta) {
  int v;
  asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(dsmem_map(smem_u32(p), cta)) : "memory");
  return v;
}

// First half: counts this warp's free pages (the loads of 16 words in flight, `meanwhile` behind the first).
template <typename F>
__device__ __forceinline__ void pool_count(const CacheParams& p, Pool& pool, uint32_t* masks, PoolShared& sh, F meanwhile) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, of_all = static_cast<int>(cluster_ctarank()) * kWarps + warp;
  constexpr int kLoads = 16;
  pool.words = p.warp_words;
  pool.first = of_all * pool.words * 32;
  pool.mask = masks + warp * pool.words;
  int count = 0;
  if (pool.words == 0) meanwhile();
#pragma unroll 1
  for (int w = 0; w < pool.words; w += kLoads) {
    int refs[kLoads];
#pragma unroll
    for (int k = 0; k < kLoads; ++k) {
      const int id = pool.first + 32 * (w + k) + lane;
      refs[k] = w + k < pool.words && id < p.num_pages ? p.page_refs[id] : 1;
    }
    if (w == 0) meanwhile();
#pragma unroll
    for (int k = 0; k < kLoads; ++k) {
      const uint32_t free = __ballot_sync(0xFFFFFFFFu, refs[k] <= 0);
      count += __popc(free);
      if (lane == 0 && w + k < pool.words) pool.mask[w + k] = free;
    }
  }
  if (lane == 0) sh.warp_free[warp] = count;
  __syncthreads();
  if (warp == 0) {
    const int all = __reduce_add_sync(0xFFFFFFFFu, sh.warp_free[lane]);
    if (lane == 0) sh.cta_free = all;
  }
}
// The free pages of a lane's word of 32, and how many are free before it: word w0 + lane of
// this warp's; *rank0 steps over all 32.
__device__ __forceinline__ uint32_t pool_word(const Pool& pool, int w0, int* rank0, int* before) {
  const int lane = threadIdx.x & 31;
  const uint32_t free = w0 + lane < pool.words ? pool.mask[w0 + lane] : 0u;
  int upto = __popc(free);
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int add = __shfl_up_sync(0xFFFFFFFFu, upto, d);
    if (lane >= d) upto += add;
  }
  *before = *rank0 + upto - __popc(free);
  *rank0 += __shfl_sync(0xFFFFFFFFu, upto, 31);
  return free;
}
// Second half, after the cluster has met.
__device__ __forceinline__ void pool_places(Pool& pool, const PoolShared& sh) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, cta = static_cast<int>(cluster_ctarank());
  const int of_cta = lane < cluster_ctas() ? remote(&sh.cta_free, lane) : 0;
  pool.free = __reduce_add_sync(0xFFFFFFFFu, of_cta);
  pool.before = __reduce_add_sync(0xFFFFFFFFu, (lane < cta ? of_cta : 0) + (lane < warp ? sh.warp_free[lane] : 0));
}

// New positions for every row, in the rows' order: row b takes q_starts[b + 1] - q_starts[b].
// The k-th page that is needed is the k-th lowest free one, so the warp that holds a free page
// finds from its rank whose it is. A row that does not fit (its places, or what is left of the pool
// behind the rows before it) takes nothing.
struct AppendRow {
  int old, n, have, want, need;
  bool fits;
};
__device__ __forceinline__ AppendRow append_row(const CacheParams& p, int old, int n) {
  AppendRow r;
  r.old = max(old, 0), r.n = n;
  const long long room = min(static_cast<long long>(p.max_pages) * p.page_size, static_cast<long long>(INT32_MAX));
  r.fits = n > 0 && static_cast<long long>(r.old) + n <= room;
  r.have = places(p, r.old);
  r.want = r.fits ? places(p, r.old + n) : r.have;
  return r;
}

__global__ void __launch_bounds__(kThreads, 1) cache_append_kernel(const __grid_constant__ CacheParams p) {
  extern __shared__ int smem[];
  __shared__ PoolShared sh;
  __shared__ int warp_need[kWarps];
  int* starts = smem;                                        // [batch + 1] first token of each row
  int* before = starts + p.batch + 1;                        // [batch + 1] pages needed before it
  int* old = before + p.batch + 1;                           // [batch]
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, cta = static_cast<int>(cluster_ctarank());
  allow_dependents_launch();
  grid_dependency_wait();
  // What each row needs; every CTA works it out for itself. A thread's first row (most have no
  // other) is looked up while the pool is: length and tokens, last page, who else holds it.
  const int per = (p.batch + kThreads - 1) / kThreads, row0 = min(tid * per, p.batch), row1 = min(row0 + per, p.batch);
  int s0 = 0, s1 = 0, len = 0, last = -1;
  AppendRow r{};
  auto look = [&](int row) {
    s0 = p.q_starts ? p.q_starts[row] : row;
    s1 = p.q_starts ? p.q_starts[row + 1] : row + 1;
    len = p.kv_lens[row];
  };
  auto look_at_table = [&](int row) {
    s0 = min(max(s0, 0), p.tokens);
    s1 = min(max(s1, s0), p.tokens);
    r = append_row(p, len, s1 - s0);
    const bool in_part = r.fits && r.old != r.have * p.page_size;      // the last page is the row's own, unless others hold it too
    last = in_part ? p.page_table[row * p.table_stride + r.have - 1] : -1;
  };
  if (row0 < row1) look(row0);
  Pool pool;
  pool_count(p, pool, reinterpret_cast<uint32_t*>(old + p.batch), sh, [&] {
    if (row0 < row1) look_at_table(row0);
  });
  int mine = 0;
  for (int row = row0; row < row1; ++row) {
    if (row > row0) {
      look(row);
      look_at_table(row);
    }
    const int need = r.want - r.have + (is_page(p, last) && p.page_refs[last] > 1);
    starts[row] = s0, old[row] = r.old, before[row] = need;
    if (row == p.batch - 1) starts[p.batch] = s1;
    mine += need;
    if (cta == 0) p.src[row] = p.dst[row] = -1;
  }
  int upto = mine;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int add = __shfl_up_sync(0xFFFFFFFFu, upto, d);
    if (lane >= d) upto += add;
  }
  if (lane == 31) warp_need[warp] = upto;
  cluster_meet();                                            // all counts, nothing given out yet
  pool_places(pool, sh);
  const int of_warp = warp_need[lane];
  const int all_need = __reduce_add_sync(0xFFFFFFFFu, of_warp);
  const int needed = min(all_need, p.tokens);                // (no more, unless q_starts decreases)
  int at = upto - mine + __reduce_add_sync(0xFFFFFFFFu, lane < warp ? of_warp : 0);
  // From here old is -1 for rows that take nothing.
  for (int row = row0; row < row1; ++row) {
    const int need = before[row];
    const AppendRow r = append_row(p, old[row], starts[row + 1] - starts[row]);
    before[row] = at;
    at += need;
    if (!r.fits || (need > 0 && at > pool.free)) old[row] = -1;
    else if (cta == 0) p.kv_lens[row] = r.old + r.n;       // (every CTA has its own copy of the old ones)
  }
  if (tid == 0) before[p.batch] = all_need;
  // The pages to give out, in their order, stand where the slots will: a row needs no more
  // pages than it has new tokens. (Few warps hold them all, so they only list them.)
  int rank0 = pool.before;
  for (int w = 0; w < pool.words && rank0 < needed; w += 32) {
    int rank;
    uint32_t free = pool_word(pool, w, &rank0, &rank);
    for (; free != 0 && rank < needed; free &= free - 1) p.slots[rank++] = pool.first + 32 * (w + lane) + __ffs(free) - 1;
  }
  cluster_meet();
  // The last row that begins at or before x, of `begins`: as many steps for everyone.
  int top = 1;
  while (2 * top < p.batch) top *= 2;
  const int step = cluster_ctas() * kThreads;
  for (int rank = cta * kThreads + tid; rank < min(needed, pool.free); rank += step) {
    const int id = p.slots[rank];
    int row = 0;
    for (int d = top; d > 0; d >>= 1)
      if (row + d < p.batch && before[row + d] <= rank) row += d;
    if (old[row] < 0) continue;
    const AppendRow r = append_row(p, old[row], starts[row + 1] - starts[row]);
    const int tail = before[row + 1] - before[row] - (r.want - r.have), k = rank - before[row];
    int* place = p.page_table + row * p.table_stride + r.have + k - tail;
    if (k < tail) {                                          // in place of a last page that others hold too
      const int shared = *place;
      p.src[row] = shared, p.dst[row] = id;
      atomicSub(p.page_refs + shared, 1);
    }
    *place = id;
    p.page_refs[id] = 1;
  }
  cluster_meet();                                            // the table is whole
  constexpr int kEach = 4;                                   // tokens of a thread in work at a time
  for (int t0 = cta * kThreads + tid; t0 < p.tokens; t0 += kEach * step) {
    int row[kEach] = {}, pos[kEach], place[kEach], id[kEach];
    for (int d = top; d > 0; d >>= 1) {
#pragma unroll
      for (int k = 0; k < kEach; ++k)
        if (row[k] + d < p.batch && starts[row[k] + d] <= t0 + k * step) row[k] += d;
    }
#pragma unroll
    for (int k = 0; k < kEach; ++k) {
      const int t = t0 + k * step, was = old[row[k]];
      const bool taken = t >= starts[row[k]] && t < starts[row[k] + 1] && was >= 0;
      pos[k] = taken ? was + t - starts[row[k]] : 0;
      place[k] = p.page_div.div(pos[k]);
      id[k] = taken ? p.page_table[row[k] * p.table_stride + place[k]] : -1;
    }
#pragma unroll
    for (int k = 0; k < kEach; ++k)
      if (t0 + k * step < p.tokens)
        p.slots[t0 + k * step] = is_page(p, id[k]) ? id[k] * p.page_size + pos[k] - place[k] * p.page_size : -1;
  }
}

// Of the U used pages those at U and above move to the free ones below U: the i-th highest of
// them to the i-th lowest of those, up to max_moves. Until the table is renumbered, a moved page's
// count says where it went (kGone + its new place), so that a place needs one look (halving in the list of moved
// pages instead, from shared memory: two meetings fewer, but 24.9 us for half a million pages, and 17.5 so).
constexpr int kGone = INT32_MIN;

__global__ void __launch_bounds__(kThreads, 1) cache_compact_kernel(const __grid_constant__ CacheParams p) {
  extern __shared__ uint32_t masks[];
  __shared__ PoolShared sh;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, cta = static_cast<int>(cluster_ctarank());
  const int all = cluster_ctas() * kThreads;
  allow_dependents_launch();
  grid_dependency_wait();
  Pool pool;
  pool_count(p, pool, masks, sh, [] {});
  for (int i = cta * kThreads + tid; i < p.max_moves; i += all) p.src[i] = p.dst[i] = -1;
  cluster_meet();
  pool_places(pool, sh);
  const int used = p.num_pages - pool.free;
  int rank0 = pool.before;
  for (int w = 0; w < pool.words; w += 32) {
    // A lane takes a word of 32 pages: `rank` are free before it, `first - rank` used.
    int rank;
    const uint32_t free = pool_word(pool, w, &rank0, &rank);
    const int first = pool.first + 32 * (w + lane), count = w + lane < pool.words ? min(max(p.num_pages - first, 0), 32) : 0;
    auto below = [&](int n) { return n <= 0 ? 0u : n >= 32 ? 0xFFFFFFFFu : (1u << n) - 1; };
    const uint32_t low = below(used - first), here = below(count);
    if (used >= first && used < first + count) sh.below = rank + __popc(free & low);
    int to = rank;
    for (uint32_t left = free & low; left != 0 && to < p.max_moves; left &= left - 1) p.dst[to++] = first + __ffs(left) - 1;
    // the used ones from U on, from the highest down
    uint32_t left = here & ~free & ~low;
    int from = used - (first + count - rank - __popc(free));   // used ones behind this word
    for (; left != 0 && from < p.max_moves; ++from) {
      const int bit = 31 - __clz(left);
      p.src[from] = first + bit;
      left ^= 1u << bit;
    }
  }
  cluster_meet();                                            // both lists are whole
  const int owner = used < p.num_pages ? used / (32 * kWarps * pool.words) : -1;
  const int moves = owner < 0 ? 0 : min(remote(&sh.below, owner), p.max_moves);
  for (int i = cta * kThreads + tid; i < moves; i += all) {
    const int from = p.src[i], to = p.dst[i];
    p.page_refs[to] = p.page_refs[from];
    p.page_refs[from] = kGone + to;
  }
  cluster_meet();
  if (moves > 0) {
    constexpr int kEach = 8;                                 // entries of a lane in flight
    const int lowest = p.src[moves - 1], chunks = (p.max_pages + 32 * kEach - 1) / (32 * kEach);
    for (int c = cta * kWarps + warp; c < p.batch * chunks; c += cluster_ctas() * kWarps) {
      const int row = c / chunks, col = (c - row * chunks) * 32 * kEach + lane;
      const int end = places(p, p.kv_lens[row]);
      int* entry = p.page_table + row * p.table_stride + col;
      int id[kEach], to[kEach];
#pragma unroll
      for (int k = 0; k < kEach; ++k) id[k] = col + 32 * k < end ? entry[32 * k] : -1;
#pragma unroll
      for (int k = 0; k < kEach; ++k) to[k] = id[k] >= lowest && id[k] < p.num_pages ? p.page_refs[id[k]] : 0;
#pragma unroll
      for (int k = 0; k < kEach; ++k)
        if (to[k] < kGone + p.num_pages) entry[32 * k] = to[k] - kGone;
    }
  }
  cluster_meet();
  for (int i = cta * kThreads + tid; i < moves; i += all) p.page_refs[p.src[i]] = 0;
}

// A launch as one cluster of `ctas` CTAs (one CTA: as it is), which may begin while the kernel
// before it runs, and waits for it.
cudaLaunchConfig_t cluster_config(int ctas, int threads, size_t smem, cudaStream_t stream, cudaLaunchAttribute (&attr)[2]) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(ctas));
  cfg.blockDim = dim3(static_cast<unsigned>(threads));
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = static_cast<unsigned>(ctas), attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = ctas > 1 ? 2 : 1;
  return cfg;
}

// How many CTAs of a kernel the current device places as one cluster, up to kMaxCtas. 8 are portable; 16 need as
// many SMs of one group, which a part of a device or another of the architecture may not have. Asked once for a device.
template <auto kKernel>
cudaError_t cluster_limit(int threads, int* most) {
  constexpr int kDevices = 64;
  thread_local int known[kDevices] = {};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < kDevices && known[dev] > 0) {
    *most = known[dev];
    return cudaSuccess;
  }
  e = ensure_smem_limit(reinterpret_cast<const void*>(kKernel), kCacheSmem);
  if (e == cudaSuccess) e = cudaFuncSetAttribute(kKernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  if (e != cudaSuccess) return e;
  cudaLaunchAttribute attr[2];
  const cudaLaunchConfig_t cfg = cluster_config(kMaxCtas, threads, kCacheSmem, nullptr, attr);
  int size = 0;
  e = cudaOccupancyMaxPotentialClusterSize(&size, kKernel, &cfg);
  if (e != cudaSuccess) return e;
  *most = std::clamp(size, 1, kMaxCtas);
  if (dev < kDevices) known[dev] = *most;
  return cudaSuccess;
}

template <auto kKernel, typename... Args>
cudaError_t launch_cluster(int ctas, int threads, size_t smem, cudaStream_t stream, const Args&... args) {
  cudaLaunchAttribute attr[2];
  const cudaLaunchConfig_t cfg = cluster_config(ctas, threads, smem, stream, attr);
  return cudaLaunchKernelEx(&cfg, kKernel, args...);
}

// A kernel over the whole pool, of which every warp looks after as many words of 32 pages, in
// `ctas` CTAs or as many as can be placed. (Fewer hold more words each: 8 take 2^23 pages, but
// not beside what an append of some 5400 rows or more keeps.)
template <auto kKernel>
cudaError_t launch_pool(CacheParams p, int ctas, size_t smem, cudaStream_t stream) {
  int most = 0;
  const cudaError_t e = cluster_limit<kKernel>(kThreads, &most);
  if (e != cudaSuccess) return e;
  ctas = std::min(ctas, p.most_ctas > 0 ? std::min(p.most_ctas, most) : most);
  const int per = 32 * ctas * kWarps;
  p.warp_words = (p.num_pages + per - 1) / per;
  smem += static_cast<size_t>(p.warp_words) * kWarps * 4;
  if (smem > kCacheSmem) return cudaErrorNotSupported;
  return launch_cluster<kKernel>(ctas, kThreads, smem, stream, p);
}

// CTAs by pages, table entries (read once: a quarter of a page's work) and tokens (four). Of the GPU's time in
// a graph, with 1, 4, 8 and 16 CTAs: a token each for 16 rows in 5200 pages 6.8, 8.4, 8.6, 9.6 us; for 31 in 20400
// 10.2, 10.2, 10.5, 11.5; 62 in 40400 11.8, 9.8, 10.0, 10.9; 124 in 80500 16.0, 12.1, 10.5, 11.3; 124 in 160900 26.6, 15.2,
// 13.5, 12.5. 2593 tokens in 20400 pages 11.3, 10.9, 11.1, 11.9. Compaction of 20400 pages, 16000 entries 8.4,
// 9.0, 9.2, 9.9; 40400 and 32000 11.9, 9.0, 9.0, 10.4; 80500 and 64000 18.0, 10.4, 8.7, 10.0; 160900 and 128000 29, 14.4, 10.6, 10.0.
int ctas_for(const CacheParams& p, long long entries, int tokens) {
  const long long work = p.num_pages + entries / 4 + 4ll * tokens;
  return work <= 28 * 1024 ? 1 : work <= 64 * 1024 ? 4 : work <= 128 * 1024 ? 8 : kMaxCtas;
}

}  // namespace

cudaError_t launch_cache_copy(const CacheCopyParams& p, int caches, int pairs, bool dense, cudaStream_t stream) {
  const dim3 grid(static_cast<unsigned>(pairs * p.blocks), static_cast<unsigned>(caches));
  if (dense) cache_copy_kernel<true><<<grid, kCopyThreads, 0, stream>>>(p);
  else cache_copy_kernel<false><<<grid, kCopyThreads, 0, stream>>>(p);
  return cudaGetLastError();
}
int cache_copy_blocks(int pieces) { return (pieces + kCopyThreads * kCopyVecs - 1) / (kCopyThreads * kCopyVecs); }

cudaError_t launch_cache_fork(const CacheParams& p, cudaStream_t stream) {
  // Up to eight places for a thread of sixteen CTAs: those are one cluster, in one launch, if they can be placed. Otherwise a CTA
  // takes eight columns, a 32-byte sector of each row, and a second launch writes the lengths. One launch and two, of the GPU in
  // a graph and among others, where the host bounds: 16200 places 2.9 and 3.5 us, 9-11 and 12.4; 64400 places 5.9 and
  // 3.9, 9-11 and 13; 128800 places 9.4 and 4.5, 12.5 and 12.5.
  const size_t rows = 2 * static_cast<size_t>(p.batch);
  auto bytes = [&](int cols_log2) { return (rows + (static_cast<size_t>(p.batch) << cols_log2)) * 4; };
  int cols_log2 = 3;
  while (kMaxCtas << cols_log2 < p.max_pages) ++cols_log2;
  if (static_cast<size_t>(p.batch) << cols_log2 <= 8 * kForkThreads) {
    int ctas = 1, most = 0;
    while (ctas << cols_log2 < p.max_pages) ctas *= 2;
    const cudaError_t e = cluster_limit<cache_fork_kernel<true>>(kForkThreads, &most);
    if (e != cudaSuccess) return e;
    if (ctas <= (p.most_ctas > 0 ? std::min(p.most_ctas, most) : most))
      return launch_cluster<cache_fork_kernel<true>>(ctas, kForkThreads, bytes(cols_log2), stream, p, cols_log2);
  }
  cols_log2 = 3;
  while (bytes(cols_log2) > kCacheSmem) --cols_log2;
  const int ctas = std::max(1, (p.max_pages + (1 << cols_log2) - 1) >> cols_log2);     // (without columns: for the lengths)
  cudaError_t e = ensure_smem_limit(reinterpret_cast<const void*>(cache_fork_kernel<false>), kCacheSmem);
  if (e == cudaSuccess)
    e = launch_dependent(cache_fork_kernel<false>, ctas, kForkThreads, static_cast<int>(bytes(cols_log2)), stream, p, cols_log2);
  if (e == cudaSuccess) e = launch_dependent(cache_fork_lens_kernel, 1, kLensThreads, 0, stream, p);
  return e;
}

cudaError_t launch_cache_append(const CacheParams& p, cudaStream_t stream) {
  const int ctas = ctas_for(p, 0, p.tokens);
  return launch_pool<cache_append_kernel>(p, ctas, (3 * static_cast<size_t>(p.batch) + 2) * 4, stream);
}

cudaError_t launch_cache_truncate(const CacheParams& p, cudaStream_t stream) {
  return launch_dependent(cache_truncate_kernel, p.batch, kCutThreads, 0, stream, p);
}

cudaError_t launch_cache_compact(const CacheParams& p, cudaStream_t stream) {
  const int ctas = ctas_for(p, static_cast<long long>(p.batch) * p.max_pages, 0);
  return launch_pool<cache_compact_kernel>(p, ctas, 0, stream);
}

}  // namespace kaio
