// Attention of many rows over a paged cache (chunks of new tokens) on the
// tensor cores. The rule of the visible keys, the line of work and the joining
// of split items are in paged_attention.cuh; an item has up to 256 rows (tokens x
// query heads of one K/V head), a unit is 128 keys.
//
// For each half of 128 rows and each key tile:
//   S = Q K^T          tcgen05.mma, Q and K in shared memory, S (f32) in TMEM
//   P = exp2(c S - m)  one thread per row: S from TMEM, P (16 bit) over S in TMEM
//   O += P V           tcgen05.mma, P from TMEM, V in shared memory, O (f32) in TMEM
// with the online softmax of paged_decode.cu in its lazy form: the reference m of
// a row is renewed, and O and the sum rescaled, only when the maximum has grown
// by more than 2^8, so weights stay below 256 (an f16 holds 65504) and a renewal
// is rare; sums are of the unrounded f32 weights.
//
// What bounds it: the tensor cores. 256 rows make each K and V tile that the TMA
// brings serve two products of 128 rows, and the two halves take turns: while the
// softmax of one half runs, the tensor cores work for the other. TMEM is full:
// two S and two O of 128 columns. The softmax warps rescale O and write the
// results themselves (both are rare), so eight of twelve warps share nearly all
// registers and every softmax thread keeps its whole row of S (128 values) in them.
//
// Issuing is half the work: on the thread that issues MMAs a wait on an mbarrier
// or a commit takes 150-300 cycles, and one thread for both halves took 5100 cycles
// a unit for 2048 of products. So each half has an issuing warp of its own; per unit it
// waits for the tiles while the softmax runs, then for P (in two parts, so that the
// product starts with the first), issues PV and the next QK back to back, and makes
// one commit. What that commit implies (the product before it is done) the softmax
// warps pass on: they release the K and V stages with plain arrivals.
//
// Warps 0-3 and 4-7: the softmax of the halves; 8, 9: their MMAs; 10, 11: K and V
// tiles by TMA, one box per page and 64 columns (pages of 16 to 1024 positions),
// pages that no row sees filled with zeros by an out-of-range coordinate. Rows of V
// that no row of the item sees are zeroed in shared memory before use: a weight of
// zero must not meet whatever the slot holds. The next item's Q is fetched as soon
// as the last QK has read this one's, and its first QK runs while O is written.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>
#include <cstdint>

#include "paged_attention.cuh"

namespace kaio {
namespace {

__device__ unsigned g_chunk_err;

constexpr int kRows = 256;
constexpr int kHalf = 128;
constexpr int kKeys = 128;
constexpr int kSoftmaxWarps = 8, kSoftmaxThreads = 32 * kSoftmaxWarps;
constexpr int kMmaWarp = 8, kLoadWarp = 10;   // and the one after each
constexpr int kThreads = 384;
// Registers a thread: 384 threads start with 168; 256 x 224 + 128 x 56 is the same total.
constexpr int kSoftmaxRegs = 224, kOtherRegs = 56;
// Named barriers (0 is __syncthreads): all softmax warps; those of a half.
constexpr int kBarAll = 1, kBarHalf = 2;
constexpr int kMinUnits = 4;
constexpr float kLazy = 8.f;            // growth of the maximum (log2) that renews the reference
using Walk = PagedWalk<kRows, kKeys>;
using Span = PagedSpan<kKeys>;

template <int kDim> struct Shape {
  static constexpr int kBoxBytes = kKeys * 128;                 // 128 rows of 64 columns
  static constexpr int kBoxes = kDim / 64;
  static constexpr int kTile = kBoxes * kBoxBytes;              // Q half, K tile or V tile
  static constexpr int kKStages = kDim == 128 ? 3 : 5, kVStages = kDim == 128 ? 2 : 5;
  static constexpr uint32_t kS = 0, kO = 256;                   // TMEM columns: S at 0 and 128, O at 256 and 256 + kDim
};

// A place in the line and what one half's softmax needs of it, worked out ahead.
struct Item : Walk {
  int plain0, plain1;    // units that every row of the half sees whole (tiles of sinks are left to the mask)
  bool mine, keys;       // the half has rows; they see something
  __device__ __forceinline__ void look(const PagedParams& p, int half) {
    if (b >= p.batch) {
      mine = keys = false;
      return;
    }
    const Span span(p, s, row0(), row1(p));
    const int rows = row1(p) - row0();
    mine = rows > kHalf * half;
    keys = span.hi > 0;
    const int h0 = row0() + kHalf * half, h1 = min(h0 + kHalf, row0() + rows) - 1;
    const int all_hi = PagedRow(p, s, h0).hi, all_lo = PagedRow(p, s, h1).lo;
    // tiles [t0, t1) are seen whole; in units, the run's first tile comes last
    const int t0 = (all_lo + kKeys - 1) / kKeys - span.lo_tile, t1 = min(all_hi / kKeys - span.lo_tile, span.run);
    plain0 = span.lo > 0 ? max(t0, 1) - 1 : t0;
    plain1 = span.lo > 0 ? t1 - 1 : t1;
  }
};

// What the warps share besides the tiles.
template <int kDim> struct Control {
  uint64_t q_full[2], s_full[2], p_full[2][2], o_done[2], start;
  uint64_t k_full[Shape<kDim>::kKStages], k_empty[Shape<kDim>::kKStages];
  uint64_t v_full[Shape<kDim>::kVStages], v_empty[Shape<kDim>::kVStages], mma_done[2];
  Walk walks[4];                     // places in the line of the MMA and load warps
  Item items[2][3];                  // of each half's softmax: this item, the next and the one after
  PagedShare share;
  float row_lse[kRows];
  uint32_t tmem_base;
  int abort_flag, last_one;
};
template <int kDim>
constexpr int kSmem = (2 + Shape<kDim>::kKStages + Shape<kDim>::kVStages) * Shape<kDim>::kTile +
                      static_cast<int>(sizeof(Control<kDim>));
static_assert(kSmem<128> <= 232448 && kSmem<64> <= 232448, "shared memory of one CTA");

template <typename T> struct Type;
template <> struct Type<__half> {
  static constexpr uint32_t kFormat = 0;
  static __device__ __forceinline__ uint32_t pack(float lo, float hi) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
};
template <> struct Type<__nv_bfloat16> {
  static constexpr uint32_t kFormat = 1;
  static __device__ __forceinline__ uint32_t pack(float lo, float hi) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
};
template <typename T>
__host__ __device__ constexpr uint32_t idesc(int n, bool b_mn) {
  return idesc_f16_f32(kHalf, n, false, b_mn) | (Type<T>::kFormat << 7) | (Type<T>::kFormat << 10);
}

__device__ __forceinline__ void tma_load_4d(void* dst, const CUtensorMap* map, uint64_t* bar, int c0, int c1, int c2,
                                            int c3) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5, %6}], [%2];" ::"r"(smem_u32(dst)),
      "l"(map), "r"(smem_u32(bar)), "r"(c0), "r"(c1), "r"(c2), "r"(c3)
      : "memory");
}

template <int kRegs> __device__ __forceinline__ void more_registers() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegs));
}
template <int kRegs> __device__ __forceinline__ void fewer_registers() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegs));
}

__device__ __forceinline__ int volatile_lane() {
  int l;
  asm volatile("mov.u32 %0, %%laneid;" : "=r"(l));
  return l;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
// Two f32 at a time.
__device__ __forceinline__ uint64_t pair(float a, float b) {
  uint64_t d;
  asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "f"(a), "f"(b));
  return d;
}
__device__ __forceinline__ float2 unpair(uint64_t v) {
  float2 d;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(d.x), "=f"(d.y) : "l"(v));
  return d;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
// 32 bytes to global memory; half of them at a time where they may not be aligned.
__device__ __forceinline__ void store32(void* p, const uint32_t (&v)[8], bool aligned) {
  if (aligned) {
    asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "r"(v[0]), "r"(v[1]), "r"(v[2]),
                 "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
                 : "memory");
  } else {
    reinterpret_cast<uint4*>(p)[0] = make_uint4(v[0], v[1], v[2], v[3]);
    reinterpret_cast<uint4*>(p)[1] = make_uint4(v[4], v[5], v[6], v[7]);
  }
}

struct ChunkParams {
  PagedParams p;
  bool out32;                         // rows of out are whole, aligned 32-byte pieces
  int k_heads_first, v_heads_first;   // order of a map's middle dimensions: heads before slots
};

template <typename T, int kDim>
__global__ void __launch_bounds__(kThreads, 1)
    paged_chunk_kernel(const __grid_constant__ CUtensorMap k_map, const __grid_constant__ CUtensorMap v_map,
                       const __grid_constant__ ChunkParams cp) {
  using S = Shape<kDim>;
  const PagedParams& p = cp.p;
  // (no static shared memory: the 1024-byte aligned tiles start at its beginning)
  extern __shared__ __align__(1024) unsigned char smem[];
  unsigned char* q_smem = smem;
  unsigned char* k_ring = smem + 2 * S::kTile;
  unsigned char* v_ring = k_ring + S::kKStages * S::kTile;
  Control<kDim>& ctl = *reinterpret_cast<Control<kDim>*>(v_ring + S::kVStages * S::kTile);

  {
    PagedShare sh;
    if (!paged_share<kRows, kKeys, kThreads>(p, blockIdx.x, gridDim.x, kMinUnits,
                                             reinterpret_cast<long long*>(smem), &ctl.walks[0], &sh))
      return;
    if (threadIdx.x == 0) ctl.share = sh;
    if (threadIdx.x > 0 && threadIdx.x < 4) ctl.walks[threadIdx.x] = ctl.walks[0];
    if (threadIdx.x >= 4 && threadIdx.x < 6) {
      const int half = threadIdx.x - 4;
      Item item;
      static_cast<Walk&>(item) = ctl.walks[0];
      item.look(p, half);
      ctl.items[half][0] = item;
      item.next_item(p);
      item.look(p, half);
      ctl.items[half][1] = item;
    }
  }

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  volatile int* abort = &ctl.abort_flag;
  if (threadIdx.x == 0) {
    for (int h = 0; h < 2; ++h) {
      mbar_init(&ctl.q_full[h], 4);
      mbar_init(&ctl.s_full[h], 1);
      mbar_init(&ctl.p_full[h][0], 5);         // four softmax warps, and the other half's issuing warp
      mbar_init(&ctl.p_full[h][1], 4);
      mbar_init(&ctl.o_done[h], 1);
      mbar_init(&ctl.mma_done[h], 1);
    }
    for (int i = 0; i < S::kKStages; ++i) {
      mbar_init(&ctl.k_full[i], 1);
      mbar_init(&ctl.k_empty[i], 2);
    }
    for (int i = 0; i < S::kVStages; ++i) {
      mbar_init(&ctl.v_full[i], 1);
      mbar_init(&ctl.v_empty[i], 2);
    }
    mbar_init(&ctl.start, 1);
    ctl.abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == kMmaWarp) {
    tmem_alloc(&ctl.tmem_base, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = ctl.tmem_base;
  auto next_item = [&](Walk& to) {
    __syncwarp();
    if (lane == 0) to.next_item(p);
    __syncwarp();
  };
  bool ok = true;
  auto wait = [&](uint64_t* bar, uint32_t parity) {
    return ok = ok && __all_sync(0xFFFFFFFFu, mbar_wait(bar, parity, abort, &g_chunk_err));
  };
  uint32_t unit_count = 0;      // units before this item: unit n has K stage n % kKStages, V stage n % kVStages

  if (warp >= kLoadWarp) {
    fewer_registers<kOtherRegs>();
    // ------------------------------------------------------------ K, V tiles
    Walk& w = ctl.walks[warp - kMmaWarp];
    const bool is_v = warp > kLoadWarp;
    const uint32_t stages = is_v ? S::kVStages : S::kKStages;
    uint64_t* full = is_v ? ctl.v_full : ctl.k_full;
    uint64_t* empty = is_v ? ctl.v_empty : ctl.k_empty;
    unsigned char* ring = is_v ? v_ring : k_ring;
    const CUtensorMap* map = is_v ? &v_map : &k_map;
    const bool heads_first = is_v ? cp.v_heads_first : cp.k_heads_first;
    const int shift = min(p.page_shift, 7);
    const int boxes = kKeys >> shift, box_keys = 1 << shift;
    const int page_mask = (1 << p.page_shift) - 1;
    uint32_t stage = 0, phase = 0;
    while (ok && w.at < ctl.share.end) {
      const Span span(p, w.s, w.row0(), w.row1(p));
      const int u1 = static_cast<int>(min(static_cast<long long>(w.units), w.unit + (ctl.share.end - w.at)));
      const int* table = p.table + w.b * p.table_stride;
      const int head = w.h;
      auto page_of = [&](int u) {
        int id = p.num_pages;                             // out of range: the box is filled with zeros
        if (lane < boxes && u < u1) {
          const int k0 = span.key0(u) + lane * box_keys;
          if (k0 < span.hi && (k0 + box_keys > span.lo || k0 < span.first)) id = table[k0 >> p.page_shift];
          if (id < 0 || id > p.num_pages) id = p.num_pages;
        }
        return id;
      };
      if (span.hi > 0) {
        int id = page_of(w.unit);
        for (int u = w.unit; u < u1; ++u) {
          const int slot = (span.key0(u) + lane * box_keys) & page_mask;
          const int next = page_of(u + 1);
          if (!wait(&empty[stage], phase ^ 1)) break;
          if (lane == 0) mbar_arrive_expect_tx(&full[stage], S::kTile);
          __syncwarp();
          ++unit_count;
          if (lane < boxes) {
            unsigned char* dst = ring + stage * S::kTile + lane * box_keys * 128;
            const int c1 = heads_first ? head : slot, c2 = heads_first ? slot : head;
#pragma unroll
            for (int b = 0; b < S::kBoxes; ++b)
              tma_load_4d(dst + b * S::kBoxBytes, map, &full[stage], 64 * b, c1, c2, id);
          }
          if (++stage == stages) stage = 0, phase ^= 1;
          id = next;
        }
      }
      if (u1 < w.units) break;
      next_item(w);
    }
    // Every copy has landed before the CTA may exit: the last fill of each stage.
    for (uint32_t i = 0; i < stages && i < unit_count; ++i)
      mbar_wait_drain(&full[(unit_count - 1 - i) % stages], ((unit_count - 1 - i) / stages) & 1, &g_chunk_err);
    __syncwarp();
  } else if (warp >= kMmaWarp) {
    fewer_registers<kOtherRegs>();
    // ------------------------------------------------------------------- MMA
    Walk& w = ctl.walks[warp - kMmaWarp];
    constexpr uint32_t kQk = idesc<T>(kKeys, false), kPv = idesc<T>(kDim, true);
    const int half = warp - kMmaWarp;
    const uint32_t s_tmem = tmem + S::kS + 128 * half, o_tmem = tmem + S::kO + kDim * half;
    // descriptors of the tiles' first 16 columns (K) or keys (V); addresses are in units of 16 bytes
    const uint64_t dq = sdesc_sw128(smem_u32(q_smem + half * S::kTile), 16, 1024);
    const uint64_t dk0 = sdesc_sw128(smem_u32(k_ring), 16, 1024);
    const uint64_t dv0 = sdesc_sw128(smem_u32(v_ring), S::kBoxBytes, 1024);
    uint32_t q_phase = 0, p_phase = 0, start_phase = 0;
    // Two halves take strict turns at the tensor cores. Left to themselves they fall
    // into step, and then both wait for products and compute softmaxes at the same
    // time. A turn is one more arrival on the barrier of P, given by the other half's
    // warp once its batch (PV, then QK) is nearly issued; a half alone gives its own.
    auto grant = [&](int h) { mbar_arrive(&ctl.p_full[h][0]); };
    auto qk = [&](uint32_t n, int grant_to) {
      if (lane == 0) {
        const uint64_t dk = dk0 + (n % S::kKStages) * (S::kTile >> 4);
#pragma unroll
        for (int ks = 0; ks < kDim / 16; ++ks) {
          if (ks == kDim / 16 - 4 && grant_to >= 0) grant(grant_to);
          const uint32_t off = ((ks >> 2) * S::kBoxBytes + (ks & 3) * 32) >> 4;
          umma_ss(s_tmem, dq + off, dk + off, kQk, ks != 0);
        }
        umma_commit(&ctl.s_full[half]);
      }
    };
    while (ok && w.at < ctl.share.end) {
      const Span span(p, w.s, w.row0(), w.row1(p));
      const int u0 = w.unit;
      const int u1 = static_cast<int>(min(static_cast<long long>(w.units), u0 + (ctl.share.end - w.at)));
      const bool both = w.row1(p) - w.row0() > kHalf;
      if (span.hi > 0 && w.row1(p) - w.row0() > kHalf * half) {
        uint32_t n = unit_count;
        if (!wait(&ctl.k_full[n % S::kKStages], (n / S::kKStages) & 1)) break;
        if (!wait(&ctl.q_full[half], q_phase)) break;
        q_phase ^= 1;
        // Half 1 begins after half 0 has begun the same item: it must not grant turns of an earlier one.
        if (half == 1) {
          if (!wait(&ctl.start, start_phase)) break;
          start_phase ^= 1;
        }
        tc_fence_after();
        qk(n, half == 1 || !both ? 0 : -1);
        if (half == 0 && both && lane == 0) mbar_arrive(&ctl.start);
        for (int u = u0; u < u1; ++u, ++n) {
          const bool more = u + 1 < u1;
          if (!wait(&ctl.v_full[n % S::kVStages], (n / S::kVStages) & 1)) break;
          unsigned char* v = v_ring + (n % S::kVStages) * S::kTile;
          const int k0 = span.key0(u);
          if (k0 + kKeys > span.hi || (k0 < span.lo && k0 + kKeys > span.first)) {
            // Zero the rows of V that no row of the item sees: [from, to), and those past hi
            // (both halves' warps do, with the same values).
            const int from = max(span.first - k0, 0), to = min(max(span.lo - k0, from), kKeys);
            auto zero = [&](int r0, int r1) {
              for (int i = 8 * r0 + lane; i < 8 * r1; i += 32)
#pragma unroll
                for (int b = 0; b < S::kBoxes; ++b)
                  *reinterpret_cast<uint4*>(v + b * S::kBoxBytes + i * 16) = make_uint4(0, 0, 0, 0);
            };
            zero(from, to);
            zero(max(min(span.hi - k0, kKeys), 0), kKeys);
            fence_proxy_async_smem();
            __syncwarp();
          }
          if (more && !wait(&ctl.k_full[(n + 1) % S::kKStages], ((n + 1) / S::kKStages) & 1)) break;
          const uint64_t dv = dv0 + (n % S::kVStages) * (S::kTile >> 4);
#pragma unroll
          for (int part = 0; part < 2; ++part) {
            if (!wait(&ctl.p_full[half][part], p_phase)) break;
            tc_fence_after();
            if (lane == 0) {
#pragma unroll
              for (int ks = 4 * part; ks < 4 * part + 4; ++ks)
                umma_ts(o_tmem, s_tmem + 8 * ks, dv + ks * 128, kPv, u != u0 || ks != 0);
            }
          }
          if (!ok) break;
          p_phase ^= 1;
          if (more) {
            qk(n + 1, both ? half ^ 1 : 0);
          } else if (lane == 0) {
            if (both && half == 0) grant(1);
            umma_commit(&ctl.o_done[half]);
          }
        }
        if (!ok) break;
      } else if (span.hi > 0) {
        // No rows of this half: it still takes every tile in turn and releases it. A
        // wait tells a phase from its neighbours only, so nobody may skip ahead.
        uint32_t n = unit_count;
        for (int u = u0; u < u1; ++u, ++n) {
          if (!wait(&ctl.k_full[n % S::kKStages], (n / S::kKStages) & 1)) break;
          if (lane == 0) mbar_arrive(&ctl.k_empty[n % S::kKStages]);
          if (!wait(&ctl.v_full[n % S::kVStages], (n / S::kVStages) & 1)) break;
          if (lane == 0) mbar_arrive(&ctl.v_empty[n % S::kVStages]);
        }
        if (!ok) break;
      }
      if (span.hi > 0) unit_count += u1 - u0;
      if (u1 < w.units) break;
      next_item(w);
    }
    // Every MMA has completed before TMEM is released.
    if (lane == 0) {
      umma_commit(&ctl.mma_done[half]);
      mbar_wait_drain(&ctl.mma_done[half], 0, &g_chunk_err);
    }
    __syncwarp();
  } else {
    more_registers<kSoftmaxRegs>();
    // --------------------------------------------------------------- softmax
    const int half = warp >> 2, of_half = warp & 3;
    const int my_row = 32 * warp + lane;                   // of the item's 256
    const uint32_t lanes = static_cast<uint32_t>(32 * of_half) << 16;
    const uint32_t s_tmem = tmem + lanes + S::kS + 128 * half, o_tmem = tmem + lanes + S::kO + kDim * half;
    // The scale is applied after the mask (-inf) and the maximum, so it has to be
    // positive: a negative one turns Q's signs, a zero makes Q zero.
    const float scale = p.scale_log2 == 0.f ? 1.f : fabsf(p.scale_log2);
    uint32_t tile_phase = 0, o_phase = 0;
    bool q_sent = false;                                   // this item's Q is already on its way

    // Q rows of this warp: global -> 128B-swizzled shared memory, asynchronously; rows past the item's are zero.
    // (Their lane comes from a volatile read, which keeps their addresses out of the registers of the loop below.)
    constexpr int kChunks = kDim / 8;
    auto q_at = [&](int rl, int q_chunk) {
      return q_smem + half * S::kTile + (q_chunk >> 3) * S::kBoxBytes + rl * 128 + (((q_chunk & 7) ^ (rl & 7)) << 4);
    };
    auto fetch_q = [&](const Walk& it) {
      const int ln = volatile_lane(), q_chunk = ln % kChunks;
      const int r0 = it.row0(), rows = it.row1(p) - r0;
      // this lane's first row as token and query head of the group, then steps of kStep rows
      constexpr int kStep = 32 / kChunks;
      int rl = 32 * of_half + ln / kChunks;
      const int first = r0 + kHalf * half + rl, t0 = p.group_div.div(first);
      int g = first - t0 * p.group;
      const T* src = static_cast<const T*>(p.q) + (it.s.q0 + t0) * p.q_ts + (it.h * p.group + g) * p.q_hs + q_chunk * 8;
      const long long wrap = p.q_ts - p.group * p.q_hs;
      const int end = q_chunk * 8 < p.dim && p.scale_log2 != 0.f ? rows - kHalf * half : 0;
#pragma unroll 4
      for (int i = 0; i < 32; i += kStep) {
        cp_async16(q_at(rl, q_chunk), rl < end ? src : static_cast<const T*>(p.q), rl < end ? 16 : 0);
        rl += kStep;
        src += kStep * p.q_hs;
        for (g += kStep; g >= p.group; g -= p.group) src += wrap;
      }
    };
    auto send_q = [&] {
      asm volatile("cp.async.wait_all;" ::: "memory");
      if (p.scale_log2 < 0.f) {                            // every lane turns the signs of what it fetched
        const int ln = volatile_lane();
        for (int i = 0; i < 32; i += 32 / kChunks) {
          uint4* v = reinterpret_cast<uint4*>(q_at(32 * of_half + i + ln / kChunks, ln % kChunks));
          v->x ^= 0x80008000u, v->y ^= 0x80008000u, v->z ^= 0x80008000u, v->w ^= 0x80008000u;
        }
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&ctl.q_full[half]);
    };

    // Named barriers keep the warps together, so a warp whose wait gave up (ok is
    // false) goes through all of them too; it only no longer waits or arrives.
    for (uint32_t item = 0;; ++item) {
      const Item& w = ctl.items[half][item % 3];
      const Item& nx = ctl.items[half][(item + 1) % 3];
      if (w.at >= ctl.share.end) break;
      const Span span(p, w.s, w.row0(), w.row1(p));
      const int u0 = w.unit;
      const int u1 = static_cast<int>(min(static_cast<long long>(w.units), u0 + (ctl.share.end - w.at)));
      const int rows = w.row1(p) - w.row0();
      const bool mine = w.mine, keys = w.keys;
      bool q_next = false;
      float m = kNegInf, l = 0.f;                          // the row's reference (in units of S), this thread's sum
      if (mine && keys) {
        if (!q_sent) {
          fetch_q(w);
          send_q();
        }
        const int plain0 = w.plain0, plain1 = w.plain1;
#pragma unroll 1
        for (int u = u0; u < u1; ++u) {
          wait(&ctl.s_full[half], tile_phase);
          tc_fence_after();
          tile_phase ^= 1;
          // QK of this unit is done, and so is PV of the one before
          if (of_half == 0 && lane == 0 && ok) mbar_arrive(&ctl.k_empty[(unit_count + (u - u0)) % S::kKStages]);
          if (of_half == 1 && lane == 0 && ok && u > u0)
            mbar_arrive(&ctl.v_empty[(unit_count + (u - u0) - 1) % S::kVStages]);
          if (u + 1 == u1 && u1 == w.units) {              // Q has been read for the last time: fetch the next item's
            q_next = nx.at < ctl.share.end && nx.mine && nx.keys;
            if (q_next) fetch_q(nx);
          }
          uint32_t s[4][32];
#pragma unroll
          for (int i = 0; i < 4; ++i) tmem_ld32(s_tmem + 32 * i, s[i]);
          tmem_ld_wait();
          if (u < plain0 || u >= plain1) {
            const PagedRow vis(p, w.s, min(w.row0() + my_row, w.row1(p) - 1));
            const int k0 = span.key0(u);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              // bits of the visible ones of these 32 keys
              const int at = k0 + 32 * i;
              auto below = [&](int x) { return x <= 0 ? 0u : x >= 32 ? 0xFFFFFFFFu : (1u << x) - 1; };
              const uint32_t seen = below(vis.hi - at) & (~below(vis.lo - at) | below(p.sinks - at));
              if (__all_sync(0xFFFFFFFFu, seen == 0xFFFFFFFFu)) continue;
#pragma unroll
              for (int e = 0; e < 32; ++e)
                if (!(seen >> e & 1)) s[i][e] = __float_as_uint(kNegInf);
            }
          }
          float top8[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) top8[i] = fmaxf(__uint_as_float(s[0][2 * i]), __uint_as_float(s[0][2 * i + 1]));
#pragma unroll
          for (int i = 8; i < 64; ++i)
            top8[i & 7] = max3(top8[i & 7], __uint_as_float(s[i >> 4][2 * i & 31]), __uint_as_float(s[i >> 4][(2 * i & 31) + 1]));
          const float top = fmaxf(max3(top8[0], top8[1], top8[2]), max3(max3(top8[3], top8[4], top8[5]), top8[6], top8[7]));
          // (the first finite maximum after none needs no rescaling: O and l are zero)
          const bool renew = top > m && (m == kNegInf || (top - m) * scale > kLazy);
          if (__any_sync(0xFFFFFFFFu, renew)) {
            if (__any_sync(0xFFFFFFFFu, renew && m != kNegInf)) {
              const float f = renew ? exp2_fast((m - top) * scale) : 1.f;
              l *= f;
#pragma unroll 1
              for (int c = 0; c < kDim; c += 16) {
                uint32_t o0[8], o1[8];
                tmem_ld8(o_tmem + c, o0);
                tmem_ld8(o_tmem + c + 8, o1);
                tmem_ld_wait();
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                  o0[e] = __float_as_uint(__uint_as_float(o0[e]) * f);
                  o1[e] = __float_as_uint(__uint_as_float(o1[e]) * f);
                }
                tmem_st8(o_tmem + c, o0);
                tmem_st8(o_tmem + c + 8, o1);
              }
              tmem_st_wait();
            }
            if (renew) m = top;
          }
          const float ref = m == kNegInf ? 0.f : m * scale;
          const uint64_t scale2 = pair(scale, scale), ref2 = pair(-ref, -ref);
          uint64_t sum2[2] = {};
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            uint32_t packed[16];
#pragma unroll
            for (int e = 0; e < 32; e += 2) {
              const float2 x = unpair(fma2(pair(__uint_as_float(s[i][e]), __uint_as_float(s[i][e + 1])), scale2, ref2));
              const float a = exp2_fast(x.x), b = exp2_fast(x.y);
              sum2[i & 1] = add2(sum2[i & 1], pair(a, b));
              packed[e >> 1] = Type<T>::pack(a, b);
            }
            tmem_st16(s_tmem + 16 * i, packed);
            if (i & 1) {                                   // 64 keys of P are complete
              tmem_st_wait();
              tc_fence_before();
              __syncwarp();
              if (lane == 0 && ok) mbar_arrive(&ctl.p_full[half][i >> 1]);
            }
          }
          const float2 sa = unpair(sum2[0]), sb = unpair(sum2[1]);
          l += (sa.x + sa.y) + (sb.x + sb.y);
        }
        if (q_next) send_q();
      }
      // The line's next item but one, for all warps of the half (after the barrier below).
      if (of_half == 0 && lane == 0) {
        Item after = nx;
        if (after.at < ctl.share.end) {
          after.next_item(p);
          after.look(p, half);
        }
        ctl.items[half][(item + 2) % 3] = after;
      }
      if (mine && keys) {
        wait(&ctl.o_done[half], o_phase);
        tc_fence_after();
        o_phase ^= 1;
        if (of_half == 1 && lane == 0 && ok)
          mbar_arrive(&ctl.v_empty[(unit_count + (u1 - u0) - 1) % S::kVStages]);
      }
      if (keys) unit_count += u1 - u0;
      q_sent = q_next;

      // Results of this thread's row: O / l and m + log2 l (nothing seen: zeros, -inf).
      const bool split = u0 != 0 || u1 != w.units;
      const bool none = l == 0.f;                          // (a NaN score leaves l NaN)
      const float inv = none ? 0.f : 1.f / l;
      const bool real = mine && my_row < rows;
      const int g = w.row0() + min(my_row, rows - 1), t = p.group_div.div(g);
      const long long tok = w.s.q0 + t;
      const int head = w.h * p.group + g - t * p.group;
      const int slot = 2 * static_cast<int>(blockIdx.x) + (u0 == 0 ? 1 : 0);
      if (mine) {
        float* to_part = p.part_o + (static_cast<long long>(slot) * kRows + my_row) * kDim;
        T* to_out = static_cast<T*>(p.out) + tok * p.o_ts + head * p.o_hs;
#pragma unroll 1
        for (int c = 0; c < kDim; c += 32) {
          uint32_t o[32];
          if (keys) {
            tmem_ld32(o_tmem + c, o);
            tmem_ld_wait();
          }
#pragma unroll
          for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(none ? 0.f : __uint_as_float(o[e]) * inv);
          if (real && split) {
#pragma unroll
            for (int e = 0; e < 32; e += 8) {
              const uint32_t v[8] = {o[e], o[e + 1], o[e + 2], o[e + 3], o[e + 4], o[e + 5], o[e + 6], o[e + 7]};
              store32(to_part + c + e, v, true);
            }
          } else if (real) {
#pragma unroll
            for (int e = 0; e < 32; e += 16) {
              const int at = c + e;
              uint32_t v[8];
#pragma unroll
              for (int k = 0; k < 8; ++k)
                v[k] = Type<T>::pack(__uint_as_float(o[e + 2 * k]), __uint_as_float(o[e + 2 * k + 1]));
              if (at + 16 <= p.dim) store32(to_out + c + e, v, cp.out32);
              else if (at < p.dim) *reinterpret_cast<uint4*>(to_out + c + e) = make_uint4(v[0], v[1], v[2], v[3]);
            }
          }
          __syncwarp();
        }
        tc_fence_before();
        if (real) {
          const float lse2 = none ? kNegInf : (m == kNegInf ? 0.f : m * scale) + log2f(l);
          if (split) p.part_l[slot * kRows + my_row] = lse2;
          else if (p.lse) p.lse[tok * p.heads + head] = lse2 * kLn2;
        }
      }
      if (split) {
        // All softmax threads come here for every split item, also when a wait gave up.
        const int c0 = ctl.share.owner(w.at - u0), c1 = ctl.share.owner(w.at - u0 + w.units - 1);
        named_sync(kBarAll, kSoftmaxThreads);
        if (threadIdx.x == 0) {
          __threadfence();                                 // covers what the others wrote before the barrier
          const unsigned seen = atomicAdd(p.counters + c0, 1u);
          ctl.last_one = seen == static_cast<unsigned>(c1 - c0);
          if (ctl.last_one) p.counters[c0] = 0;
        }
        named_sync(kBarAll, kSoftmaxThreads);
        if (ctl.last_one) {
          __threadfence();
          // Each row's log-sum over all parts (one thread a row); a part then
          // weighs exp2(its own - that).
          if (my_row < rows) {
            float top = kNegInf, sum = 0.f;
#pragma unroll 4
            for (int c = c0; c <= c1; ++c) top = fmaxf(top, __ldcg(p.part_l + (2 * c + (c == c0)) * kRows + my_row));
            const float ref = top == kNegInf ? 0.f : top;
#pragma unroll 4
            for (int c = c0; c <= c1; ++c)
              sum += exp2_fast(__ldcg(p.part_l + (2 * c + (c == c0)) * kRows + my_row) - ref);
            ctl.row_lse[my_row] = sum == 0.f ? kNegInf : ref + log2f(sum);
          }
          named_sync(kBarAll, kSoftmaxThreads);
          // Eight columns a thread, so that a part's row is read and the output's
          // written in whole sectors; kBatch rows at once for loads in flight.
          constexpr int kLanes = kDim / 8, kRowStep = kSoftmaxThreads / kLanes, kBatch = 4;
          const int col = threadIdx.x % kLanes * 8;
          for (int r0 = threadIdx.x / kLanes; r0 < rows; r0 += kBatch * kRowStep) {
            float acc[kBatch][8] = {}, lse2r[kBatch];
#pragma unroll
            for (int k = 0; k < kBatch; ++k) lse2r[k] = r0 + k * kRowStep < rows ? ctl.row_lse[r0 + k * kRowStep] : kNegInf;
            for (int c = c0; c <= c1; ++c) {
              const long long from = (2 * c + (c == c0)) * kRows + r0;
#pragma unroll
              for (int k = 0; k < kBatch; ++k) {
                if (lse2r[k] == kNegInf) continue;         // past the rows, or nothing seen
                const float f = exp2_fast(__ldcg(p.part_l + from + k * kRowStep) - lse2r[k]);
                const float4* src = reinterpret_cast<const float4*>(p.part_o + (from + k * kRowStep) * kDim + col);
                const float4 a = __ldcg(src), b = __ldcg(src + 1);
                acc[k][0] += f * a.x, acc[k][1] += f * a.y, acc[k][2] += f * a.z, acc[k][3] += f * a.w;
                acc[k][4] += f * b.x, acc[k][5] += f * b.y, acc[k][6] += f * b.z, acc[k][7] += f * b.w;
              }
            }
#pragma unroll
            for (int k = 0; k < kBatch; ++k) {
              const int r = r0 + k * kRowStep;
              if (r >= rows) continue;
              const int gr = w.row0() + r, tr = p.group_div.div(gr), hr = w.h * p.group + gr - tr * p.group;
              const long long at = w.s.q0 + tr;
              uint4 v;
              v.x = Type<T>::pack(acc[k][0], acc[k][1]);
              v.y = Type<T>::pack(acc[k][2], acc[k][3]);
              v.z = Type<T>::pack(acc[k][4], acc[k][5]);
              v.w = Type<T>::pack(acc[k][6], acc[k][7]);
              if (col < p.dim)
                *reinterpret_cast<uint4*>(static_cast<T*>(p.out) + at * p.o_ts + hr * p.o_hs + col) = v;
              if (p.lse && col == 0) p.lse[at * p.heads + hr] = lse2r[k] * kLn2;
            }
          }
        }
        named_sync(kBarAll, kSoftmaxThreads);                    // ctl.last_one has been read
      }
      if (u1 < w.units) break;
      named_sync(kBarHalf + half, 128);                 // all are done with this item, and the next but one is known
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == kMmaWarp) tmem_dealloc(tmem, 512);
}

// [pages][slots][heads][dim] (strides in elements) as a 4-D map of boxes of 64
// columns x up to 128 slots of one head of one page, the middle dimensions in
// the order of their strides.
cudaError_t encode_cache(CUtensorMap* map, int* heads_first, const void* base, FloatType t, const PagedParams& p,
                         long long ps, long long ss, long long hs) {
  const uint64_t page = 1ull << p.page_shift;
  *heads_first = p.kv_heads > 1 && hs < ss;
  uint64_t dims[4] = {static_cast<uint64_t>(p.dim), page, static_cast<uint64_t>(p.kv_heads),
                      static_cast<uint64_t>(p.num_pages)};
  // the stride of a dimension of one element is never used
  uint64_t strides[3] = {static_cast<uint64_t>(ss) * 2, p.kv_heads > 1 ? static_cast<uint64_t>(hs) * 2 : 16,
                         p.num_pages > 1 ? static_cast<uint64_t>(ps) * 2 : 16};
  uint32_t box[4] = {64, static_cast<uint32_t>(std::min<uint64_t>(page, kKeys)), 1, 1};
  if (*heads_first) {
    std::swap(dims[1], dims[2]);
    std::swap(strides[0], strides[1]);
    std::swap(box[1], box[2]);
  }
  const CUresult r = encode_tensor_map(map,
                                       t == FloatType::BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                                                            : CU_TENSOR_MAP_DATA_TYPE_FLOAT16,
                                       4, base, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B);
  return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

template <typename T, int kDim>
cudaError_t launch(const CUtensorMap& km, const CUtensorMap& vm, const ChunkParams& cp, int ctas, cudaStream_t stream) {
  const cudaError_t e =
      ensure_smem_limit(reinterpret_cast<const void*>(paged_chunk_kernel<T, kDim>), kSmem<kDim>);
  if (e != cudaSuccess) return e;
  paged_chunk_kernel<T, kDim><<<ctas, kThreads, kSmem<kDim>, stream>>>(km, vm, cp);
  return cudaGetLastError();
}

}  // namespace

size_t paged_chunk_workspace_bytes(int num_sms) {
  return kPagedCounterBytes + 32 + 2 * static_cast<size_t>(num_sms) * kRows * (128 + 1) * sizeof(float);
}

cudaError_t launch_paged_chunk(FloatType t, const PagedParams& params, void* workspace, int num_sms,
                               cudaStream_t stream) {
  ChunkParams cp{};
  cp.p = params;
  PagedParams& p = cp.p;
  const int ctas = std::min(num_sms, static_cast<int>(kPagedCounterBytes / sizeof(unsigned)));
  p.counters = static_cast<unsigned*>(workspace);
  // 32-byte stores: the workspace itself is only 16-byte aligned
  p.part_o = reinterpret_cast<float*>((reinterpret_cast<uintptr_t>(workspace) + kPagedCounterBytes + 31) & ~31ull);
  cp.out32 = reinterpret_cast<uintptr_t>(p.out) % 32 == 0 && (p.tokens == 1 || p.o_ts % 16 == 0) &&
             (p.heads == 1 || p.o_hs % 16 == 0);
  p.part_l = p.part_o + static_cast<size_t>(2) * ctas * kRows * (p.dim <= 64 ? 64 : 128);
  CUtensorMap km, vm;
  cudaError_t e = encode_cache(&km, &cp.k_heads_first, p.kc, t, p, p.k_ps, p.k_ss, p.k_hs);
  if (e == cudaSuccess) e = encode_cache(&vm, &cp.v_heads_first, p.vc, t, p, p.v_ps, p.v_ss, p.v_hs);
  if (e != cudaSuccess) return e;
  if (t == FloatType::BF16)
    return p.dim <= 64 ? launch<__nv_bfloat16, 64>(km, vm, cp, ctas, stream)
                       : launch<__nv_bfloat16, 128>(km, vm, cp, ctas, stream);
  return p.dim <= 64 ? launch<__half, 64>(km, vm, cp, ctas, stream) : launch<__half, 128>(km, vm, cp, ctas, stream);
}

unsigned read_and_clear_chunk_errors() {
  unsigned v = 0;
  if (cudaMemcpyFromSymbol(&v, g_chunk_err, sizeof(v)) != cudaSuccess) return 0xFFFFFFFFu;
  const unsigned zero = 0;
  cudaMemcpyToSymbol(g_chunk_err, &zero, sizeof(zero));
  return v;
}

}  // namespace kaio
