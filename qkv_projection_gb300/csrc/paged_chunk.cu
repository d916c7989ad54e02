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
// Warps 0-3 and 4-7: the softmax of the halves; 8: MMA (10, 11 only fill its group of
// four, by which registers are shared out); 9: K and V tiles by TMA,
// one box per page and 64 columns (pages of 16 to 1024 positions), pages that no
// row sees filled with zeros by an out-of-range coordinate. Rows of V that no row
// of the item sees are zeroed in shared memory before use: a weight of zero must
// not meet whatever the slot holds.
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
constexpr int kSoftmaxThreads = 256;
constexpr int kMmaWarp = 8, kLoadWarp = 9;
constexpr int kThreads = 384;
// Registers a thread: 384 threads start with 168; 2 x 128 x 208 + 128 x 88 is the same total.
constexpr int kSoftmaxRegs = 208, kOtherRegs = 88;
constexpr int kMinUnits = 4;
constexpr float kLazy = 8.f;            // growth of the maximum (log2) that renews the reference
using Walk = PagedWalk<kRows, kKeys>;
using Span = PagedSpan<kKeys>;

template <int kDim> struct Shape {
  static constexpr int kBoxBytes = kKeys * 128;                 // 128 rows of 64 columns
  static constexpr int kBoxes = kDim / 64;
  static constexpr int kTile = kBoxes * kBoxBytes;              // Q half, K tile or V tile
  static constexpr int kStages = kDim == 128 ? 5 : 10;
  static constexpr int kSmem = (2 + kStages) * kTile + 1024;
  static constexpr uint32_t kS = 0, kO = 256;                   // TMEM columns: S at 0 and 128, O at 256 and 256 + kDim
};

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

struct ChunkParams {
  PagedParams p;
  int k_heads_first, v_heads_first;   // order of a map's middle dimensions: heads before slots
};

template <typename T, int kDim>
__global__ void __launch_bounds__(kThreads, 1)
    paged_chunk_kernel(const __grid_constant__ CUtensorMap k_map, const __grid_constant__ CUtensorMap v_map,
                       const __grid_constant__ ChunkParams cp) {
  using S = Shape<kDim>;
  const PagedParams& p = cp.p;
  extern __shared__ unsigned char smem_raw[];
  unsigned char* smem = align_smem_1024(smem_raw);
  unsigned char* q_smem = smem;
  unsigned char* ring = smem + 2 * S::kTile;
  __shared__ __align__(8) uint64_t q_full[2], s_full[2], p_full[2], o_done[2], kv_full[S::kStages],
      kv_empty[S::kStages], mma_done;
  __shared__ Walk walks[kMmaWarp + 2];      // every warp's own place in the line (in registers it would cost the softmax 20)
  __shared__ PagedShare share;
  __shared__ uint32_t tmem_base;
  __shared__ int abort_flag, last_one;

  {
    PagedShare sh;
    if (!paged_share<kRows, kKeys, kThreads>(p, blockIdx.x, gridDim.x, kMinUnits,
                                             reinterpret_cast<long long*>(smem), &walks[0], &sh))
      return;
    if (threadIdx.x == 0) share = sh;
    if (threadIdx.x > 0 && threadIdx.x < kMmaWarp + 2) walks[threadIdx.x] = walks[0];
  }

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  volatile int* abort = &abort_flag;
  if (threadIdx.x == 0) {
    for (int h = 0; h < 2; ++h) {
      mbar_init(&q_full[h], 4);
      mbar_init(&s_full[h], 1);
      mbar_init(&p_full[h], 4);
      mbar_init(&o_done[h], 1);
    }
    for (int i = 0; i < S::kStages; ++i) {
      mbar_init(&kv_full[i], 1);
      mbar_init(&kv_empty[i], 1);
    }
    mbar_init(&mma_done, 1);
    abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == kMmaWarp) {
    tmem_alloc(&tmem_base, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_base;
  Walk& w = walks[min(warp, kLoadWarp)];
  auto next_item = [&] {
    __syncwarp();
    if (lane == 0) w.next_item(p);
    __syncwarp();
  };

  if (warp == kLoadWarp) {
    fewer_registers<kOtherRegs>();
    // ------------------------------------------------------------ K, V tiles
    const int shift = min(p.page_shift, 7);
    const int boxes = kKeys >> shift, box_keys = 1 << shift;
    const int page_mask = (1 << p.page_shift) - 1;
    int stage = 0;
    uint32_t phase = 0;
    bool ok = true;
    uint32_t used = 0;                                    // stages filled at least once
    while (ok && w.at < share.end) {
      const Span span(p, w.s, w.row0(), w.row1(p));
      const int u1 = static_cast<int>(min(static_cast<long long>(w.units), w.unit + (share.end - w.at)));
      const int* table = p.table + w.b * p.table_stride;
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
        for (int u = w.unit; ok && u < u1; ++u) {
          const int slot = (span.key0(u) + lane * box_keys) & page_mask;
          const int next = page_of(u + 1);
#pragma unroll
          for (int kv = 0; kv < 2; ++kv) {
            ok = __all_sync(0xFFFFFFFFu, mbar_wait(&kv_empty[stage], phase ^ 1, abort, &g_chunk_err));
            if (!ok) break;
            if (lane == 0) mbar_arrive_expect_tx(&kv_full[stage], S::kTile);
            __syncwarp();
            used |= 1u << stage;
            if (lane < boxes) {
              unsigned char* dst = ring + stage * S::kTile + lane * box_keys * 128;
              const CUtensorMap* map = kv ? &v_map : &k_map;
              const bool heads_first = kv ? cp.v_heads_first : cp.k_heads_first;
              const int c1 = heads_first ? w.h : slot, c2 = heads_first ? slot : w.h;
#pragma unroll
              for (int b = 0; b < S::kBoxes; ++b)
                tma_load_4d(dst + b * S::kBoxBytes, map, &kv_full[stage], 64 * b, c1, c2, id);
            }
            if (++stage == S::kStages) stage = 0, phase ^= 1;
          }
          id = next;
        }
      }
      if (u1 < w.units) break;
      next_item();
    }
    // Every copy has landed before the CTA may exit.
    for (int i = 0; i < S::kStages; ++i)
      if (used >> i & 1) mbar_wait_drain(&kv_full[i], i < stage ? phase : phase ^ 1, &g_chunk_err);
    __syncwarp();
  } else if (warp == kMmaWarp) {
    fewer_registers<kOtherRegs>();
    // ------------------------------------------------------------------- MMA
    constexpr uint32_t kQk = idesc<T>(kKeys, false), kPv = idesc<T>(kDim, true);
    int stage = 0;
    uint32_t phase = 0, q_phase[2] = {}, p_phase[2] = {};
    bool ok = true;
    auto wait = [&](uint64_t* bar, uint32_t ph) {
      ok = ok && mbar_wait(bar, ph, abort, &g_chunk_err);
      ok = __all_sync(0xFFFFFFFFu, ok);
      tc_fence_after();
      return ok;
    };
    auto advance = [&](int& st, uint32_t& ph) {
      if (++st == S::kStages) st = 0, ph ^= 1;
    };
    auto qk = [&](int h, int st) {
      if (lane == 0) {
        const uint32_t sq = smem_u32(q_smem + h * S::kTile), sk = smem_u32(ring + st * S::kTile);
#pragma unroll
        for (int ks = 0; ks < kDim / 16; ++ks) {
          const uint32_t off = (ks >> 2) * S::kBoxBytes + (ks & 3) * 32;
          umma_ss(tmem + S::kS + 128 * h, sdesc_sw128(sq + off, 16, 1024), sdesc_sw128(sk + off, 16, 1024), kQk,
                  ks != 0);
        }
        umma_commit(&s_full[h]);
      }
    };
    auto pv = [&](int h, int st, bool accumulate) {
      if (lane == 0) {
        const uint32_t sv = smem_u32(ring + st * S::kTile);
#pragma unroll
        for (int ks = 0; ks < kKeys / 16; ++ks)
          umma_ts(tmem + S::kO + kDim * h, tmem + S::kS + 128 * h + 8 * ks,
                  sdesc_sw128(sv + ks * 2048, S::kBoxBytes, 1024), kPv, accumulate || ks != 0);
        umma_commit(&o_done[h]);
      }
    };
    while (ok && w.at < share.end) {
      const Span span(p, w.s, w.row0(), w.row1(p));
      const int u1 = static_cast<int>(min(static_cast<long long>(w.units), w.unit + (share.end - w.at)));
      const int halves = w.row1(p) - w.row0() > kHalf ? 2 : 1;
      if (span.hi > 0) {
        int k_stage = stage;
        if (!wait(&kv_full[k_stage], phase)) break;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          if (h >= halves || !wait(&q_full[h], q_phase[h])) break;
          q_phase[h] ^= 1;
          qk(h, k_stage);
        }
        if (!ok) break;
        if (lane == 0) umma_commit(&kv_empty[k_stage]);
        advance(stage, phase);
        for (int u = w.unit; u < u1; ++u) {
          const int v_stage = stage;
          if (!wait(&kv_full[v_stage], phase)) break;
          advance(stage, phase);
          const int k0 = span.key0(u);
          if (k0 + kKeys > span.hi || (k0 < span.lo && k0 + kKeys > span.first)) {
            // zero the rows of V that no row of the item sees
            unsigned char* v = ring + v_stage * S::kTile;
            for (int i = lane; i < kKeys * S::kBoxes * 8; i += 32) {
              const int key = (i >> 3) & (kKeys - 1), j = k0 + key;
              if (!(j < span.hi && (j >= span.lo || j < span.first)))
                *reinterpret_cast<uint4*>(v + i * 16) = make_uint4(0, 0, 0, 0);
            }
            fence_proxy_async_smem();
            __syncwarp();
          }
          const bool more = u + 1 < u1;
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            if (h >= halves || !wait(&p_full[h], p_phase[h])) break;
            p_phase[h] ^= 1;
            pv(h, v_stage, u != w.unit);
            if (h == halves - 1 && lane == 0) umma_commit(&kv_empty[v_stage]);
            if (more) {
              if (h == 0 && !wait(&kv_full[stage], phase)) break;
              qk(h, stage);
            }
          }
          if (!ok) break;
          if (more) {
            if (lane == 0) umma_commit(&kv_empty[stage]);
            advance(stage, phase);
          }
        }
        if (!ok) break;
      }
      if (u1 < w.units) break;
      next_item();
    }
    // Every MMA has completed before TMEM is released.
    if (lane == 0) {
      umma_commit(&mma_done);
      mbar_wait_drain(&mma_done, 0, &g_chunk_err);
    }
    __syncwarp();
  } else if (warp >= 8) {
    fewer_registers<kOtherRegs>();
  } else {
    more_registers<kSoftmaxRegs>();
    // --------------------------------------------------------------- softmax
    const int half = warp >> 2;
    const uint32_t lanes = static_cast<uint32_t>(32 * (warp & 3)) << 16;
    const uint32_t s_tmem = tmem + lanes + S::kS + 128 * half, o_tmem = tmem + lanes + S::kO + kDim * half;
    const int my_row = 32 * warp + lane;                   // of the item's 256
    // The scale is applied after the mask (-inf) and the maximum, so it has to be
    // positive: a negative one turns Q's signs, a zero makes Q zero.
    const float scale = p.scale_log2 == 0.f ? 1.f : fabsf(p.scale_log2);
    const uint32_t flip = p.scale_log2 < 0.f ? 0x80008000u : 0u;
    uint32_t tile_phase = 0;                               // of s_full and o_done
    bool ok = true;
    auto wait = [&](uint64_t* bar, uint32_t ph) {
      ok = __all_sync(0xFFFFFFFFu, mbar_wait(bar, ph, abort, &g_chunk_err));
      tc_fence_after();
      return ok;
    };
    while (w.at < share.end) {
      const Span span(p, w.s, w.row0(), w.row1(p));
      const int u0 = w.unit;
      const int u1 = static_cast<int>(min(static_cast<long long>(w.units), u0 + (share.end - w.at)));
      const int rows = w.row1(p) - w.row0();
      const bool mine = half == 0 || rows > kHalf;         // this half has rows
      const bool keys = span.hi > 0;
      float m = kNegInf, l = 0.f;                          // reference (in units of S) and sum
      if (mine && keys && ok) {
        {  // Q rows of this warp: global -> 128B-swizzled shared memory, rows past the item's are zero
          constexpr int kChunks = kDim / 8;
          const int chunk = lane % kChunks;
#pragma unroll 4
          for (int i = 0; i < 32; i += 32 / kChunks) {
            const int r = 32 * warp + i + lane / kChunks;
            uint4 v = make_uint4(0, 0, 0, 0);
            if (r < rows && chunk * 8 < p.dim && p.scale_log2 != 0.f) {
              const int g = w.row0() + r, t = g / p.group;
              v = *reinterpret_cast<const uint4*>(static_cast<const T*>(p.q) + (w.s.q0 + t) * p.q_ts +
                                                  (w.h * p.group + g - t * p.group) * p.q_hs + chunk * 8);
              v.x ^= flip, v.y ^= flip, v.z ^= flip, v.w ^= flip;
            }
            const int rl = r & (kHalf - 1);
            *reinterpret_cast<uint4*>(q_smem + half * S::kTile + (chunk >> 3) * S::kBoxBytes + rl * 128 +
                                      (((chunk & 7) ^ (rl & 7)) << 4)) = v;
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(&q_full[half]);
        }
        const int h0 = w.row0() + kHalf * half, h1 = min(h0 + kHalf, w.row0() + rows) - 1;
        const int all_hi = PagedRow(p, w.s, h0).hi, all_lo = PagedRow(p, w.s, h1).lo;
        const PagedRow vis(p, w.s, min(w.row0() + my_row, h1));
#pragma unroll 1
        for (int u = u0; u < u1; ++u) {
          if (!wait(&s_full[half], tile_phase)) break;
          uint32_t s[4][32];
#pragma unroll
          for (int i = 0; i < 4; ++i) tmem_ld32(s_tmem + 32 * i, s[i]);
          tmem_ld_wait();
          const int k0 = span.key0(u);
          if (!(k0 + kKeys <= all_hi && (k0 >= all_lo || k0 + kKeys <= p.sinks))) {
            const int hi = vis.hi - k0, lo = vis.lo - k0, first = p.sinks - k0;
#pragma unroll
            for (int i = 0; i < 128; ++i)
              if (!(i < hi && (i >= lo || i < first))) s[i >> 5][i & 31] = __float_as_uint(kNegInf);
          }
          float top4[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            top4[i] = __uint_as_float(s[i][0]);
#pragma unroll
            for (int e = 1; e < 32; ++e) top4[i] = fmaxf(top4[i], __uint_as_float(s[i][e]));
          }
          const float top = fmaxf(fmaxf(top4[0], top4[1]), fmaxf(top4[2], top4[3]));
          // (the first finite maximum after none needs no rescaling: O and l are zero)
          const bool renew = top > m && (m == kNegInf || (top - m) * scale > kLazy);
          if (__any_sync(0xFFFFFFFFu, renew && m != kNegInf)) {
            // the product that last wrote O has to be done
            if (!wait(&o_done[half], tile_phase ^ 1)) break;
            const float f = renew ? exp2_fast((m - top) * scale) : 1.f;
            l *= f;
#pragma unroll 1
            for (int c = 0; c < kDim; c += 32) {
              uint32_t o[32];
              tmem_ld32(o_tmem + c, o);
              tmem_ld_wait();
#pragma unroll
              for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
              tmem_st32(o_tmem + c, o);
            }
            tmem_st_wait();
          }
          if (renew) m = top;
          const float ref = m == kNegInf ? 0.f : m * scale;
          float sum[4] = {};
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            uint32_t packed[16];
#pragma unroll
            for (int e = 0; e < 32; e += 2) {
              const float a = exp2_fast(fmaf(__uint_as_float(s[i][e]), scale, -ref));
              const float b = exp2_fast(fmaf(__uint_as_float(s[i][e + 1]), scale, -ref));
              sum[i] += a + b;
              packed[e >> 1] = Type<T>::pack(a, b);
            }
            tmem_st16(s_tmem + 16 * i, packed);
          }
          l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
          tmem_st_wait();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&p_full[half]);
          tile_phase ^= 1;
        }
        if (ok) wait(&o_done[half], tile_phase ^ 1);
      }

      // Results of this thread's row: O / l and m + log2 l (nothing seen: zeros, -inf).
      const bool split = u0 != 0 || u1 != w.units;
      const bool none = l == 0.f;                          // (a NaN score leaves l NaN)
      const float inv = none ? 0.f : 1.f / l;
      const float lse2 = none ? kNegInf : (m == kNegInf ? 0.f : m * scale) + log2f(l);
      const bool real = mine && my_row < rows;
      const int g = w.row0() + min(my_row, rows - 1), t = g / p.group;
      const long long tok = w.s.q0 + t;
      const int head = w.h * p.group + g - t * p.group;
      const int slot = 2 * static_cast<int>(blockIdx.x) + (u0 == 0 ? 1 : 0);
      if (mine) {
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
            float* dst = p.part_o + (static_cast<long long>(slot) * kRows + my_row) * kDim + c;
#pragma unroll
            for (int e = 0; e < 32; e += 4)
              *reinterpret_cast<uint4*>(dst + e) = make_uint4(o[e], o[e + 1], o[e + 2], o[e + 3]);
          } else if (real) {
            T* dst = static_cast<T*>(p.out) + tok * p.o_ts + head * p.o_hs + c;
#pragma unroll
            for (int e = 0; e < 32; e += 8)
              if (c + e < p.dim) {
                uint4 v;
                uint32_t* pv = &v.x;
#pragma unroll
                for (int k = 0; k < 4; ++k)
                  pv[k] = Type<T>::pack(__uint_as_float(o[e + 2 * k]), __uint_as_float(o[e + 2 * k + 1]));
                *reinterpret_cast<uint4*>(dst + e) = v;
              }
          }
          __syncwarp();
        }
        tc_fence_before();
        if (real) {
          if (split) p.part_l[slot * kRows + my_row] = lse2;
          else if (p.lse) p.lse[tok * p.heads + head] = lse2 * kLn2;
        }
      }
      if (split) {
        // All softmax threads come here for every split item, also when a wait gave up.
        const int c0 = share.owner(w.at - u0), c1 = share.owner(w.at - u0 + w.units - 1);
        __threadfence();
        named_sync(1, kSoftmaxThreads);
        if (threadIdx.x == 0) {
          const unsigned seen = atomicAdd(p.counters + c0, 1u);
          last_one = seen == static_cast<unsigned>(c1 - c0);
          if (last_one) p.counters[c0] = 0;
        }
        named_sync(1, kSoftmaxThreads);
        if (last_one) {
          __threadfence();
          constexpr int kCols = kDim / 32;                 // columns of a lane
          for (int r = warp; r < rows; r += 8) {
            float top = kNegInf;
            for (int c = c0; c <= c1; ++c) top = fmaxf(top, __ldcg(p.part_l + (2 * c + (c == c0)) * kRows + r));
            const float ref = top == kNegInf ? 0.f : top;
            float acc[kCols] = {}, sum = 0.f;
#pragma unroll 4
            for (int c = c0; c <= c1; ++c) {
              const int from = 2 * c + (c == c0);
              const float f = exp2_fast(__ldcg(p.part_l + from * kRows + r) - ref);
              sum += f;
              const float* src = p.part_o + (static_cast<long long>(from) * kRows + r) * kDim + kCols * lane;
#pragma unroll
              for (int e = 0; e < kCols; e += 2) {
                const float2 v = __ldcg(reinterpret_cast<const float2*>(src + e));
                acc[e] += f * v.x;
                acc[e + 1] += f * v.y;
              }
            }
            const float norm = sum == 0.f ? 0.f : 1.f / sum;
            const int gr = w.row0() + r, tr = gr / p.group, hr = w.h * p.group + gr - tr * p.group;
            const long long at = w.s.q0 + tr;
            if (kCols * lane < p.dim) {
              uint32_t* dst = reinterpret_cast<uint32_t*>(static_cast<T*>(p.out) + at * p.o_ts + hr * p.o_hs + kCols * lane);
#pragma unroll
              for (int e = 0; e < kCols; e += 2) dst[e >> 1] = Type<T>::pack(acc[e] * norm, acc[e + 1] * norm);
            }
            if (p.lse && lane == 0)
              p.lse[at * p.heads + hr] = sum == 0.f ? kNegInf : (ref + log2f(sum)) * kLn2;
          }
        }
        named_sync(1, kSoftmaxThreads);                    // last_one has been read
      }
      if (u1 < w.units) break;
      next_item();
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
      ensure_smem_limit(reinterpret_cast<const void*>(paged_chunk_kernel<T, kDim>), Shape<kDim>::kSmem);
  if (e != cudaSuccess) return e;
  paged_chunk_kernel<T, kDim><<<ctas, kThreads, Shape<kDim>::kSmem, stream>>>(km, vm, cp);
  return cudaGetLastError();
}

}  // namespace

size_t paged_chunk_workspace_bytes(int num_sms) {
  return kPagedCounterBytes + 2 * static_cast<size_t>(num_sms) * kRows * (128 + 1) * sizeof(float);
}

cudaError_t launch_paged_chunk(FloatType t, const PagedParams& params, void* workspace, int num_sms,
                               cudaStream_t stream) {
  ChunkParams cp{};
  cp.p = params;
  PagedParams& p = cp.p;
  const int ctas = std::min(num_sms, static_cast<int>(kPagedCounterBytes / sizeof(unsigned)));
  p.counters = static_cast<unsigned*>(workspace);
  p.part_o = reinterpret_cast<float*>(static_cast<char*>(workspace) + kPagedCounterBytes);
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
