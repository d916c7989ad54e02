// Attention of many rows over a paged cache (chunks of new tokens) on the
// tensor cores. The rule of the visible keys, the line of work and the joining
// of split items are in paged_attention.cuh; an item has up to 256 rows (tokens x
// query heads of one K/V head), a unit is 128 keys.
//
// For each half of 128 rows and each key tile:
//   S = Q K^T          tcgen05.mma, Q and K in shared memory, S (f32) in TMEM
//   P = exp2(c S - m)  one thread per row: S from TMEM, P (16 bit) over S in TMEM
//   O += P V           tcgen05.mma, P from TMEM, V in shared memory, O (f32) in TMEM
// with the online softmax of paged_decode.cuh in its lazy form: the reference m of
// a row is renewed, and O and the sum rescaled, only when the maximum has grown
// by more than 2^8, so a renewal is rare; sums are of the unrounded f32 weights. In f16
// the exponents are raised by 7 (for the reason in paged_decode.cuh): the largest weight
// of a row lies between 2^7 and 2^15, of the 65504 that fit, and what is lost 2^-32 or
// more below it.
//
// What bounds it: many rows, the chain of each half (below); few rows, the bytes of K
// and V. 256 rows make each K and V tile that the TMA brings serve two products of
// 128 rows. The two halves take strict turns at the tensor cores: while the softmax
// of one runs, they work for the other. A unit of 256 rows takes 3100-3250 cycles for
// 2016 of products; the rest is the way from product to softmax to product, with one
// wait and one commit of 150-300 cycles each. TMEM is full (two S and two O of 128
// columns), so there is no third half to fill the gap. 4096 tokens over 16384 keys,
// 32 heads on 8 of 128: 726-750 us with the power limit, 1.28-1.33 PFLOP/s, 0.66-0.68 of
// what the measured library product reaches in a burst, 0.74-0.77 of it sustained
// (680-690 us on a GPU that kept a higher clock, beside which the figures of other forms below were taken).
//
// Registers: the softmax warps rescale O and write the results themselves (both are
// rare), so eight of twelve warps share nearly all registers (216 a thread, 72 for the
// others) and every softmax thread keeps its whole row of S, 128 values, in them. The
// loop is sensitive to that: some hundred bytes of spills cost 8-20 %.
//
// Issuing is half the work: on the thread that issues MMAs a wait on an mbarrier
// or a commit takes 150-300 cycles, and one thread for both halves took 5100 cycles
// a unit for 2016 of products. So each half has an issuing warp of its own; per unit it
// waits for the tiles while the softmax runs, then for P (in two parts, so that the
// product starts with the first), issues PV and the next QK back to back, and makes
// one commit. What that commit implies (the product before it is done) the softmax
// warps pass on: they release the K and V stages with plain arrivals. A turn rides on
// the barrier of P as one more arrival.
//
// Few rows (single tokens among chunks, short chunks): up to 128 rows and at least two
// units make the halves a pair, which takes every other unit each on the same rows and
// joins in tensor memory at the end: 2600 cycles a unit, 43 GB/s for each SM, which is
// the memory's rate. Such a unit counts 3 in the line of work, one of 256 rows 4 (a mixed
// step of 31 single tokens and 512 new ones: 136 us with equal counts, 121 us so, 114 with
// the cost of an item).
//
// Scores of other forms (a cap, a bias that grows with distance, documents, prefixes; each a
// kernel of its own): what a row's scores go through happens in the same registers, between the
// load from TMEM and the maximum. The chain of a half is longer by it, so these are bound by the softmax warps:
// - a cap costs a second exponential and an eighth of a reciprocal a score. The exponential unit takes 4 cycles
//   a warp's exponential, 9 a reciprocal: 9 cycles a score where 4 were (a quarter: 10, and 11 measured for the whole sequence
//   alone, 12.3 with one warp); two halves' 128 scores then fill 2330 of a unit's 5000 cycles, 1280 more than without a cap. The
//   unit takes 1700 more; what the rest is (36-40 bytes a thread that spill, halves that compute at the same
//   time) has not been told apart. 4096 tokens over 16384: 1050 us with a quarter, 1033-1040 with an eighth, 0.93 PFLOP/s; with
//   a window of 4096 365 us, and 235 without a cap.
// - a bias makes the nearest keys the heaviest, so the tiles of its kernels run from the last to the first: from the
//   first on, most tiles would raise a steep head's maximum and rescale O (4096 tokens over 16384: 1100 us so, 788 in reverse,
//   773-784 since pieces that a warp sees nothing of are not worked on). Slopes below zero, whose heaviest keys are the
//   farthest, meet their tiles from that wrong end: 923-939 us. Without causal order what lies right of a row goes through the
//   short loop below: 1020 us, and 740 without slopes. With a cap, too, 1228 us; 76-84 bytes a thread spill there.
// - units with hidden keys, and those a bias does not fall evenly over (the row's own place lies inside), go
//   through one short loop of 32 keys at a time, in place in TMEM, before the rest. Unrolled over 128 in registers it cost a
//   prompt of documents 147 us, rolled 128-130: such items have five units on average, and code that is fetched anew runs at 5 cycles an
//   instruction. With a cap the loop also takes scores of more than 5 caps.
// Measured and not kept: the weights through shared memory, so that the next product of Q and K runs behind the
// softmax (no wait for it left, but 400 cycles more for each 64 keys' stores and fence, and the issuing thread late: with a cap
// 1214 us, with slopes 970); units in parts of 64 keys with a product each (1262); two threads a row (1200); halves held half a
// unit's time apart (1160); waits polled (1233); the next unit's scores in two products of 64 keys, the first behind
// this one's softmax or between its two products (1103 to 1155, with slopes 813 to 846: a product of 64 keys takes the tensor
// cores about as long as one of 128).
//
// Warps 0-3 and 4-7: the softmax of the halves; 8, 9: their MMAs; 10: works out the
// jobs (items, or this CTA's part of one) a few ahead and loads K; 11: loads V. Tiles
// come by TMA, one box per page and 64 columns (pages of 16 to 1024 positions), pages
// that no row sees filled with zeros by an out-of-range coordinate. Rows of V that no
// row of the item sees are zeroed in shared memory before use: a weight of zero must not
// meet whatever the slot holds. The next item's Q is fetched as soon as the last QK has
// read this one's, and its first QK runs while O is written.
//
// Split items: the CTA that is last joins the parts in their order. Up to three parts it
// joins from its own tensor memory and the workspace; more only from the workspace, with
// ten loads of a thread in flight (one after another a part took 6000 cycles).
//
// A CTA whose wait gave up still counts itself in at every split item of its share, so
// that the last one to come clears the counter, as always: the outputs are lost, the
// workspace is not.
#pragma once

#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>
#include <cstdint>
#include <type_traits>

#include "paged_attention.cuh"

namespace kaio {
namespace {

__device__ unsigned g_chunk_err;

constexpr int kRows = 256;
constexpr int kHalf = 128;
constexpr int kKeys = 128;
constexpr int kSoftmaxWarps = 8;
constexpr int kMmaWarp = 8, kLoadWarp = 10;   // and the one after each
constexpr int kThreads = 384;
// Registers a thread: 384 threads start with 168; 256 x 216 + 128 x 72 is the same total.
constexpr int kSoftmaxRegs = 216, kOtherRegs = 72;
constexpr int kFewParts = 3;            // parts up to which the last CTA joins the others' with its own still in tensor memory
constexpr float kLazy = 8.f;            // growth of the maximum (log2) that renews the reference
// An item besides its units takes 7500 cycles, two units' time, whatever its length (2574
// new tokens, 32/8 heads, tiles of 1 to 21 units: 85 us with items of up to 16 whole and free
// of cost, 71 us so). A part is worth a unit: 100 tokens over 9000 keys with 32/8 heads take
// 59 us, and 61 us with 0.6 units, 20 over 60000 with 8/1 79 and 81, with two units 84.
template <bool kWithScores>
struct Work {
  static constexpr bool kScored = kWithScores;
  static constexpr int kRows = 256, kFewRows = 128, kKeys = 128;
  static constexpr int kCost = 4, kSmallRows = 128, kSmallCost = 3, kItemCost = 8, kSnap = 16;
  static constexpr int kWhole = 16, kJoin = 6, kWholeOfMany = 0;
  static constexpr float kPartWorth = 1.f;
};

template <int kDim> struct Shape {
  static constexpr int kBoxBytes = kKeys * 128;                 // 128 rows of 64 columns
  static constexpr int kBoxes = kDim / 64;
  static constexpr int kTile = kBoxes * kBoxBytes;              // Q half, K tile or V tile
  static constexpr int kKStages = kDim == 128 ? 3 : 5, kVStages = kDim == 128 ? 2 : 5;
  static constexpr uint32_t kS = 0, kO = 256;                   // TMEM columns: S at 0 and 128, O at 256 and 256 + kDim
};

// How the halves share an item: one has up to 128 rows and works alone; both have
// rows; or up to 128 rows and at least two units are worked on by both, who take
// every other unit and join their results at the end (few rows against many keys are
// bound by one half's chain of product, softmax and product).
enum class Mode : int { kEnd, kNoKeys, kAlone, kBoth, kPair };

// An item, or this CTA's part of one, as the load warp works it out for all others.
template <bool kScored>
struct Job {
  Mode mode;
  int q0, row0, rows, h, b;           // first token of the sequence; rows of the item; K/V head, sequence
  PagedSeq s;
  int u0, u1;                         // units of this part
  int plain0[2], plain1[2];           // units that every row of a half sees whole (tiles of sinks are left to the mask)
  int c0, c1;                         // the CTAs that share the item, if more than one do
  bool split;                         // only a part of the item
  PagedSpan<kKeys, kScored> span;
};
constexpr int kJobs = 4;

// What the warps share besides the tiles.
template <int kDim, bool kScored> struct Control {
  uint64_t q_full[2], s_full[2], p_full[2][2], o_done[2], start, meet;
  uint64_t k_full[Shape<kDim>::kKStages], k_empty[Shape<kDim>::kKStages];
  uint64_t v_full[Shape<kDim>::kVStages], v_empty[Shape<kDim>::kVStages], mma_done[2];
  uint64_t job_full[kJobs], job_empty[kJobs];
  PagedWalk<Work<kScored>> place;
  PagedShare share;
  Job<kScored> jobs[kJobs];
  float row_lse[kRows], row_mul[kRows];
  uint32_t tmem_base, planned, entered;   // jobs worked out, and begun by thread 0
  int abort_flag, last_one;
};
template <int kDim, bool kScored>
constexpr int kSmem = (2 + Shape<kDim>::kKStages + Shape<kDim>::kVStages) * Shape<kDim>::kTile +
                      static_cast<int>(sizeof(Control<kDim, kScored>));
static_assert(kSmem<128, true> <= 232448 && kSmem<64, true> <= 232448, "shared memory of one CTA");

template <typename T> struct Type;
template <> struct Type<__half> {
  static constexpr uint32_t kFormat = 0;
  static constexpr int kShift = 7;
  static __device__ __forceinline__ uint32_t pack(float lo, float hi) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
};
template <> struct Type<__nv_bfloat16> {
  static constexpr uint32_t kFormat = 1;
  static constexpr int kShift = 0;
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
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ float min_nan(float a, float b) {
  float d;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
  return d;
}
// cap tanh(x) = cap - 2 cap / (1 + exp(2x)): four scores become -1 / (1 + exp2(c s)), c = 2 log2(e)
// scale / cap. The factor 2 cap goes into what follows, the constant cap into the log-sum. The four
// share a reciprocal (1/a = bcd / abcd, known as batch inversion), so c s is at most kCapRange, where the tanh is 1 - 2^-29.
// Errors, in 2^-23: of exp2 (approximate to 2^-22.5, its argument rounded twice) 0.8 after the
// quotient's slope of at most a quarter, of the reciprocal, the sum and the products 3.5 (4.5 where eight share one); so a
// score is off by at most 24 * 2^-24 caps, and far less where it is large, since the results are small there.
constexpr float kCapRange = 30.f;
__device__ __forceinline__ void cap4(uint32_t* s, float c) {
  const uint64_t c2 = pair(c, c), minus1 = pair(-1.f, -1.f);
  const float2 y = unpair(mul2(pair(__uint_as_float(s[0]), __uint_as_float(s[1])), c2));
  const float2 z = unpair(mul2(pair(__uint_as_float(s[2]), __uint_as_float(s[3])), c2));
  const uint64_t a = fma2(pair(exp2_fast(y.x), exp2_fast(y.y)), minus1, minus1);
  const uint64_t b = fma2(pair(exp2_fast(z.x), exp2_fast(z.y)), minus1, minus1);
  const float2 ab = unpair(mul2(a, b));
  const float all = rcp_fast(ab.x * ab.y);
  const uint64_t inv = pair(all * ab.y, all * ab.x);       // 1 / (a b) of either half
  const float2 u = unpair(mul2(inv, b)), v = unpair(mul2(inv, a));
  s[0] = __float_as_uint(u.x), s[1] = __float_as_uint(u.y);
  s[2] = __float_as_uint(v.x), s[3] = __float_as_uint(v.y);
}
// The same of 128 scores of at most kCapRange / 2, of which eight share a reciprocal. Sixteen a
// step and three steps in work at a time: what one waits for (the exponentials, the reciprocal) the others' work covers.
__device__ __forceinline__ void cap128(uint32_t (&s)[4][32], float c) {
  uint64_t ab[2][4], abcd[2][2];
  float inv[2][2];
  auto at = [&](int e) -> uint32_t& { return s[e >> 5][e & 31]; };
  auto get = [&](int e) { return pair(__uint_as_float(at(e)), __uint_as_float(at(e + 1))); };
  auto set = [&](int e, uint64_t v) {
    const float2 x = unpair(v);
    at(e) = __float_as_uint(x.x), at(e + 1) = __float_as_uint(x.y);
  };
  const uint64_t c2 = pair(c, c), minus1 = pair(-1.f, -1.f);
#pragma unroll
  for (int b = 0; b < 10; ++b) {
    if (b < 8) {
#pragma unroll
      for (int e = 16 * b; e < 16 * b + 16; e += 2) {
        const float2 y = unpair(mul2(get(e), c2));
        set(e, pair(exp2_fast(y.x), exp2_fast(y.y)));
      }
    }
    if (b >= 1 && b < 9) {
      const int now = (b - 1) & 1;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int e = 16 * (b - 1) + 4 * k;
        set(e, fma2(get(e), minus1, minus1));
        set(e + 2, fma2(get(e + 2), minus1, minus1));
        ab[now][k] = mul2(get(e), get(e + 2));
      }
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        abcd[now][k] = mul2(ab[now][2 * k], ab[now][2 * k + 1]);
        const float2 x = unpair(abcd[now][k]);
        inv[now][k] = rcp_fast(x.x * x.y);
      }
    }
    if (b >= 2) {
      const int now = b & 1;
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const float2 x = unpair(abcd[now][k]);
        const uint64_t of_all = pair(inv[now][k] * x.y, inv[now][k] * x.x);
        const uint64_t of_ab = mul2(of_all, ab[now][2 * k + 1]), of_cd = mul2(of_all, ab[now][2 * k]);
        const int e = 16 * (b - 2) + 8 * k;
        const uint64_t first = get(e), third = get(e + 4);
        set(e, mul2(of_ab, get(e + 2)));
        set(e + 2, mul2(of_ab, first));
        set(e + 4, mul2(of_cd, get(e + 6)));
        set(e + 6, mul2(of_cd, third));
      }
    }
  }
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
  unsigned long long wait_ns;         // limit of a wait; used where kLimited
};

// kLimited: waits are limited to wait_ns (a test of the path that gives up).
template <typename T, int kDim, Form kForm, bool kLimited>
__global__ void __launch_bounds__(kThreads, 1)
    paged_chunk_kernel(const __grid_constant__ CUtensorMap k_map, const __grid_constant__ CUtensorMap v_map,
                       const __grid_constant__ ChunkParams cp) {
  constexpr bool kScored = kForm != Form::kPlain, kCapped = is_capped(kForm), kDistance = has_distance(kForm);
  using S = Shape<kDim>;
  using Walk = PagedWalk<Work<kScored>>;
  using Span = typename Walk::Span;
  using Row = PagedRow<kScored>;
  using Job = Job<kScored>;
  const PagedParams& p = cp.p;
  // (no static shared memory: the 1024-byte aligned tiles start at its beginning)
  extern __shared__ __align__(1024) unsigned char smem[];
  unsigned char* q_smem = smem;
  unsigned char* k_ring = smem + 2 * S::kTile;
  unsigned char* v_ring = k_ring + S::kKStages * S::kTile;
  Control<kDim, kScored>& ctl = *reinterpret_cast<Control<kDim, kScored>*>(v_ring + S::kVStages * S::kTile);

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
    mbar_init(&ctl.meet, kSoftmaxWarps);
    for (int i = 0; i < kJobs; ++i) {
      mbar_init(&ctl.job_full[i], 1);
      mbar_init(&ctl.job_empty[i], kSoftmaxWarps + 3);      // the softmax, MMA and V warps
    }
    ctl.abort_flag = 0;
    ctl.planned = ctl.entered = 0;
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
  allow_dependents_launch();
  grid_dependency_wait();
  // An empty share goes on with a plan of no jobs.
  bool any;
  {
    PagedShare sh;
    any = paged_share<kThreads>(p, blockIdx.x, gridDim.x, reinterpret_cast<long long*>(smem), &ctl.place, &sh);
    if (any && threadIdx.x == 0) ctl.share = sh;
    __syncthreads();
  }
  bool ok = true;
  auto wait = [&](uint64_t* bar, uint32_t parity) {
    auto done = [&] {
      if constexpr (kLimited) return mbar_wait_lim(bar, parity, abort, &g_chunk_err, cp.wait_ns);
      else return mbar_wait(bar, parity, abort, &g_chunk_err);
    };
    return ok = ok && __all_sync(0xFFFFFFFFu, done());
  };
  // All warps are out of their jobs.
  auto all_out = [&] { asm volatile("bar.sync 1, %0;" ::"n"(kThreads) : "memory"); };
  uint32_t unit_count = 0;      // units before this job: unit n has K stage n % kKStages, V stage n % kVStages
  auto job_ready = [&](uint32_t k) -> const Job& {
    wait(&ctl.job_full[k % kJobs], (k / kJobs) & 1);
    return ctl.jobs[k % kJobs];
  };
  auto job_done = [&](uint32_t k) {
    __syncwarp();
    if (lane == 0 && ok) mbar_arrive(&ctl.job_empty[k % kJobs]);
  };

  if (warp >= kLoadWarp) {
    fewer_registers<kOtherRegs>();
    // ---------------------------------------------------- jobs, K and V tiles
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
    for (uint32_t k = 0;; ++k) {
      if (!is_v) {
        // work out the next job, while the others are still busy with earlier ones
        if (!wait(&ctl.job_empty[k % kJobs], ((k / kJobs) & 1) ^ 1)) break;
        if (lane == 0) {
          Walk& w = ctl.place;
          Job& job = ctl.jobs[k % kJobs];
          const int u0 = any ? w.unit : 0, u1 = any && w.b < p.batch ? w.cut(ctl.share.end, ctl.share) : 0;
          if (u1 <= u0) {
            job.mode = Mode::kEnd;
          } else {
            const int row0 = w.row0(), rows = w.row1(p) - row0;
            const Span span(p, w.s, row0, row0 + rows, paged_doc<kScored>(p, w.s, row0));
            job.mode = span.hi == 0 ? Mode::kNoKeys : rows > kHalf ? Mode::kBoth : u1 - u0 > 1 ? Mode::kPair : Mode::kAlone;
            job.q0 = w.s.q0, job.row0 = row0, job.rows = rows, job.h = w.h, job.b = w.b, job.s = w.s;
            job.u0 = u0, job.u1 = u1, job.span = span;
            job.split = u0 != 0 || u1 != w.units;
            const bool last = u1 == w.units;
#pragma unroll 1
            for (int half = 0; half < 2; ++half) {
              const int h0 = row0 + (rows > kHalf ? kHalf * half : 0), h1 = min(h0 + kHalf, row0 + rows) - 1;
              const Row top(p, w.s, h0, 0), bottom(p, w.s, h1, paged_doc<kScored>(p, w.s, h1));
              const int all_hi = top.hi, all_lo = max(bottom.lo, bottom.from);
              // tiles [t0, t1) are seen whole; in units, the run's first tile comes last (or all in reverse)
              const int t0 = (all_lo + kKeys - 1) / kKeys - span.lo_tile, t1 = min(all_hi / kKeys - span.lo_tile, span.run);
              job.plain0[half] = span.back() ? span.run - t1 : span.lo > 0 ? max(t0, 1) - 1 : t0;
              job.plain1[half] = span.back() ? span.run - t0 : span.lo > 0 ? t1 - 1 : t1;
            }
            if (job.split) {
              job.c0 = w.first_owner(ctl.share);
              job.c1 = w.last_owner(ctl.share);
            }
            if (last) w.next_item(p);
            else w.unit = w.units;                         // the share ends here
          }
          if (job.mode != Mode::kEnd) ctl.planned = k + 1;
          mbar_arrive(&ctl.job_full[k % kJobs]);
        }
        __syncwarp();
      } else {
        job_ready(k);
        if (!ok) break;
      }
      const Job& job = ctl.jobs[k % kJobs];
      const Mode mode = job.mode;
      if (mode == Mode::kEnd) break;
      if (mode != Mode::kNoKeys) {
        const int* table = p.table + job.b * p.table_stride;
        const int head = job.h, u1 = job.u1;
        const Span span = job.span;
        auto page_of = [&](int u) {
          int id = p.num_pages;                             // out of range: the box is filled with zeros
          if (lane < boxes && u < u1) {
            const int k0 = span.key0(u) + lane * box_keys;
            const bool in_first = k0 < span.first && (!kScored || k0 + box_keys > span.from);
            if (k0 < span.hi && (k0 + box_keys > span.lo || in_first)) id = table[k0 >> p.page_shift];
            if (id < 0 || id > p.num_pages) id = p.num_pages;
          }
          return id;
        };
        int id = page_of(job.u0);
        for (int u = job.u0; u < u1; ++u) {
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
      if (!ok) break;
      if (is_v) job_done(k);
    }
    // Every copy has landed before the CTA may exit: the last fill of each stage.
    for (uint32_t i = 0; i < stages && i < unit_count; ++i)
      mbar_wait_drain(&full[(unit_count - 1 - i) % stages], ((unit_count - 1 - i) / stages) & 1, &g_chunk_err);
    __syncwarp();
    all_out();
    if (!is_v && lane == 0 && *abort) {
      // The split items that thread 0 did not come to: those of planned jobs, and the last
      // one of the share. (The first job is planned before any wait that can give up, so no
      // other is left that begins before the share.)
      auto count_in = [&](int c0, int c1) {
        if (atomicAdd(p.counters + c0, 1u) == static_cast<unsigned>(c1 - c0)) p.counters[c0] = 0;
      };
      for (uint32_t k = ctl.entered; k < ctl.planned; ++k) {
        const Job& job = ctl.jobs[k % kJobs];
        if (job.split) count_in(job.c0, job.c1);
      }
      Walk& w = ctl.place;
      while (any && w.b < p.batch && w.unit == 0) {
        const int u1 = w.cut(ctl.share.end, ctl.share);
        if (u1 < w.units) {
          if (u1 > 0) count_in(blockIdx.x, w.last_owner(ctl.share));
          break;
        }
        w.next_item(p);
      }
    }
  } else if (warp >= kMmaWarp) {
    fewer_registers<kOtherRegs>();
    // ------------------------------------------------------------------- MMA
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
    // The tiles that this half does not use it still takes in turn and releases (kn,
    // vn: the next of each): a wait tells a phase from its neighbours only, so nobody may skip ahead.
    uint32_t kn = 0, vn = 0;
    auto pass_k = [&](uint32_t upto) {
      for (; ok && kn < upto; ++kn)
        if (wait(&ctl.k_full[kn % S::kKStages], (kn / S::kKStages) & 1) && lane == 0)
          mbar_arrive(&ctl.k_empty[kn % S::kKStages]);
    };
    auto pass_v = [&](uint32_t upto) {
      for (; ok && vn < upto; ++vn)
        if (wait(&ctl.v_full[vn % S::kVStages], (vn / S::kVStages) & 1) && lane == 0)
          mbar_arrive(&ctl.v_empty[vn % S::kVStages]);
    };
    auto take_k = [&](uint32_t n) {
      pass_k(n);
      ++kn;
      return wait(&ctl.k_full[n % S::kKStages], (n / S::kKStages) & 1);
    };
    auto take_v = [&](uint32_t n) {
      pass_v(n);
      ++vn;
      return wait(&ctl.v_full[n % S::kVStages], (n / S::kVStages) & 1);
    };
    for (uint32_t k = 0;; ++k) {
      const Job& job = job_ready(k);
      if (!ok || job.mode == Mode::kEnd) break;
      const Mode mode = job.mode;
      if (mode != Mode::kNoKeys) {
        const uint32_t end = unit_count + (job.u1 - job.u0);
        if (half == 0 || mode != Mode::kAlone) {
          const bool both = mode == Mode::kBoth;
          const uint32_t step = mode == Mode::kPair ? 2 : 1;
          const uint32_t n0 = unit_count + (mode == Mode::kPair ? half : 0);
          if (!take_k(n0) || !wait(&ctl.q_full[half], q_phase)) break;
          q_phase ^= 1;
          // Half 1 begins after half 0 has begun the same item: it must not grant turns of an earlier one.
          if (both && half == 1) {
            if (!wait(&ctl.start, start_phase)) break;
            start_phase ^= 1;
          }
          tc_fence_after();
          qk(n0, !both ? half : half == 1 ? 0 : -1);
          if (both && half == 0 && lane == 0) mbar_arrive(&ctl.start);
#pragma unroll 1
          for (uint32_t n = n0; n < end; n += step) {
            const bool more = n + step < end;
            if (!take_v(n)) break;
            const int k0 = job.span.key0(job.u0 + static_cast<int>(n - unit_count));
            const int lo = job.span.lo, hi = job.span.hi, first = job.span.first, seen0 = kScored ? job.span.from : 0;
            if (k0 + kKeys > hi || (k0 < lo && (k0 + kKeys > first || (kScored && k0 < seen0)))) {
              // Zero the rows of V that no row of the item sees: [from, to), those past hi and
              // those before the first document (where both halves use the tile, both do, with the same values).
              unsigned char* v = v_ring + (n % S::kVStages) * S::kTile;
              const int from = max(first - k0, 0), to = min(max(lo - k0, from), kKeys);
              const int from2 = max(min(hi - k0, kKeys), to), before = kScored ? min(seen0, lo) - k0 : 0;
              for (int i = lane; i < 8 * kKeys; i += 32)
                if ((i >= 8 * from && i < 8 * to) || i >= 8 * from2 || (kScored && i < 8 * before)) {
#pragma unroll
                  for (int b = 0; b < S::kBoxes; ++b)
                    *reinterpret_cast<uint4*>(v + b * S::kBoxBytes + i * 16) = make_uint4(0, 0, 0, 0);
                }
              fence_proxy_async_smem();
              __syncwarp();
            }
            if (more && !take_k(n + step)) break;
            const uint64_t dv = dv0 + (n % S::kVStages) * (S::kTile >> 4);
#pragma unroll
            for (int part = 0; part < 2; ++part) {
              if (!wait(&ctl.p_full[half][part], p_phase)) break;
              tc_fence_after();
              if (lane == 0) {
#pragma unroll
                for (int ks = 4 * part; ks < 4 * part + 4; ++ks)
                  umma_ts(o_tmem, s_tmem + 8 * ks, dv + ks * 128, kPv, n != n0 || ks != 0);
              }
            }
            if (!ok) break;
            p_phase ^= 1;
            if (more) {
              qk(n + step, both ? half ^ 1 : half);
            } else if (lane == 0) {
              if (both && half == 0) grant(1);
              umma_commit(&ctl.o_done[half]);
            }
          }
          if (!ok) break;
        }
        while (ok && vn < end) {
          pass_k(min(vn + 1, end));
          pass_v(vn + 1);
        }
        pass_k(end);
        if (!ok) break;
        unit_count = end;
      }
      job_done(k);
    }
    // Every MMA has completed before TMEM is released.
    if (lane == 0) {
      umma_commit(&ctl.mma_done[half]);
      mbar_wait_drain(&ctl.mma_done[half], 0, &g_chunk_err);
    }
    __syncwarp();
    all_out();
  } else {
    more_registers<kSoftmaxRegs>();
    // --------------------------------------------------------------- softmax
    const int half = warp >> 2, of_half = warp & 3;
    const uint32_t lanes = static_cast<uint32_t>(32 * of_half) << 16;
    const uint32_t s_tmem = tmem + lanes + S::kS + 128 * half, o_tmem = tmem + lanes + S::kO + kDim * half;
    // The scale is applied after the mask (-inf) and the maximum, so it has to be
    // positive: a negative one turns Q's signs, a zero makes Q zero.
    // (Scored: of what the passes over the scores below leave in their place.)
    const float raw_scale = p.scale_log2 == 0.f ? 1.f : fabsf(p.scale_log2);
    const float cap_scale = kCapped ? 2.f * p.cap_log2 : raw_scale;
    const float scale = kDistance ? 1.f : cap_scale;
    const float most = kCapped ? kCapRange / p.cap_in : 0.f;
    // What a row's scores, times the scale, get added as exponents of its weights. Rounded
    // down, so that no weight is above 2^(kLazy + kShift) at any size of the reference.
    constexpr int kShift = Type<T>::kShift;
    auto addend = [&](float m) { return m == kNegInf ? kShift : __fmaf_rd(-m, scale, kShift); };
    uint32_t tile_phase = 0, o_phase = 0;
    bool q_sent = false;                                   // this item's Q is already on its way

    // Q rows of this warp: global -> 128B-swizzled shared memory, asynchronously; rows past the item's are zero.
    // (Their lane comes from a volatile read, which keeps their addresses out of the registers of the loop below.)
    constexpr int kChunks = kDim / 8;
    auto q_at = [&](int rl, int q_chunk) {
      return q_smem + half * S::kTile + (q_chunk >> 3) * S::kBoxBytes + rl * 128 + (((q_chunk & 7) ^ (rl & 7)) << 4);
    };
    auto fetch_q = [&](const Job& it) {
      const int ln = volatile_lane(), q_chunk = ln % kChunks;
      const int base = it.mode == Mode::kBoth ? kHalf * half : 0;
      // this lane's first row as token and query head of the group, then steps of kStep rows
      constexpr int kStep = 32 / kChunks;
      int rl = 32 * of_half + ln / kChunks;
      const int first = it.row0 + base + rl, t0 = p.group_div.div(first);
      int g = first - t0 * p.group;
      const T* src = static_cast<const T*>(p.q) + (it.q0 + t0) * p.q_ts + (it.h * p.group + g) * p.q_hs + q_chunk * 8;
      const long long wrap = p.q_ts - p.group * p.q_hs;
      const int end = q_chunk * 8 < p.dim && p.scale_log2 != 0.f ? it.rows - base : 0;
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

    auto works = [&](Mode mode) { return mode >= Mode::kBoth || (mode == Mode::kAlone && half == 0); };

    // All softmax warps meet where halves or parts are joined (on an mbarrier, whose wait is bounded).
    uint32_t meet_phase = 0;
    auto meet = [&] {
      __syncwarp();
      if (lane == 0 && ok) mbar_arrive(&ctl.meet);
      wait(&ctl.meet, meet_phase);
      meet_phase ^= 1;
    };
    // A warp whose wait gave up (ok is false) runs on to the end of its job without
    // waiting or arriving anywhere, and leaves.
    for (uint32_t k = 0;; ++k) {
      const Job& w = job_ready(k);
      if (!ok || w.mode == Mode::kEnd) break;
      if (threadIdx.x == 0) ctl.entered = k + 1;
      const Mode mode = w.mode;
      const int rows = w.rows, n_units = w.u1 - w.u0;
      const int my_row = (rows > kHalf ? kHalf * half : 0) + 32 * of_half + lane;   // of the item's 256
      const bool mine = works(mode) || (mode == Mode::kNoKeys && rows > kHalf * half);
      const bool keys = mode != Mode::kNoKeys;
      bool q_next = false;
      // Of an item in few parts the CTA that finds all others written is the last.
      auto look_for_others = [&] {
        if (w.split && threadIdx.x == 0) {
          unsigned seen;
          asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(seen) : "l"(p.counters + w.c0) : "memory");
          ctl.last_one = w.c1 - w.c0 < kFewParts && seen == static_cast<unsigned>(w.c1 - w.c0);
        }
      };
      float m = kNegInf, l = 0.f;                          // the row's reference (in units of S) and sum
      int doc = 0;                                         // of this thread's row: its document's begin,
      int my_pos = 0;                                      // its place,
      float slope = 0.f;                                   // and what a score gains with each position to the right
      if (kScored) {
        const int r = w.row0 + min(my_row, rows - 1);
        doc = paged_doc<kScored>(p, w.s, r);
        my_pos = w.s.kv - w.s.n + p.group_div.div(r);
        if (kDistance) slope = slope_log2(p.slopes[w.h * p.group + r - p.group_div.div(r) * p.group]);
      }
      if (works(mode)) {
        if (!q_sent) {
          fetch_q(w);
          send_q();
        }
        const int plain0 = w.plain0[half], plain1 = w.plain1[half], u1 = w.u1;
        const int step = mode == Mode::kPair ? 2 : 1, first_unit = w.u0 + (mode == Mode::kPair ? half : 0);
        uint32_t n = unit_count + (mode == Mode::kPair ? half : 0);
#pragma unroll 1
        for (int u = first_unit; u < u1; u += step, n += step) {
          wait(&ctl.s_full[half], tile_phase);
          tc_fence_after();
          tile_phase ^= 1;
          // QK of this unit is done, and so is PV of the one before
          if (of_half == 0 && lane == 0 && ok) mbar_arrive(&ctl.k_empty[n % S::kKStages]);
          if (of_half == 1 && lane == 0 && ok && u > first_unit) mbar_arrive(&ctl.v_empty[(n - step) % S::kVStages]);
          if (u + step >= u1) {                            // Q has been read for the last time: fetch the next job's
            const Job& nx = job_ready(k + 1);
            q_next = ok && works(nx.mode);
            if (q_next) fetch_q(nx);
          }
          // Bits of those of 32 keys from `at` on that a row sees; the others' scores to -inf.
          auto seen_of = [&](const Row& vis, int at) {
            auto below = [&](int x) { return x <= 0 ? 0u : x >= 32 ? 0xFFFFFFFFu : (1u << x) - 1; };
            uint32_t seen = below(vis.hi - at) & (~below(vis.lo - at) | below(vis.first - at));
            if (kScored) seen &= ~below(vis.from - at);
            return seen;
          };
          auto hide = [&](uint32_t seen, uint32_t (&x)[32]) {
            if (__all_sync(0xFFFFFFFFu, seen == 0xFFFFFFFFu)) return;
#pragma unroll
            for (int e = 0; e < 32; ++e)
              if (!(seen >> e & 1)) x[e] = __float_as_uint(kNegInf);
          };
          uint32_t s[4][32];
          auto load = [&] {
#pragma unroll
            for (int i = 0; i < 4; ++i) tmem_ld32(s_tmem + 32 * i, s[i]);
            tmem_ld_wait();
          };
          auto top_of = [&] {
            float top8[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) top8[i] = fmaxf(__uint_as_float(s[0][2 * i]), __uint_as_float(s[0][2 * i + 1]));
#pragma unroll
            for (int i = 8; i < 64; ++i)
              top8[i & 7] = max3(top8[i & 7], __uint_as_float(s[i >> 4][2 * i & 31]), __uint_as_float(s[i >> 4][(2 * i & 31) + 1]));
            return fmaxf(max3(top8[0], top8[1], top8[2]), max3(max3(top8[3], top8[4], top8[5]), top8[6], top8[7]));
          };
          float top = kNegInf;
          if constexpr (!kScored) {
            load();
            if (u < plain0 || u >= plain1) {
              const Row vis(p, w.s, w.row0 + min(my_row, rows - 1), 0);
              const int k0 = w.span.key0(u);
#pragma unroll
              for (int i = 0; i < 4; ++i) hide(seen_of(vis, k0 + 32 * i), s[i]);
            }
            top = top_of();
          } else {
            const bool masked = u < plain0 || u >= plain1;
            const int key0 = kDistance ? w.span.key0(u) : 0;
            // Units with hidden keys, and those that a bias does not fall evenly over, go 32 keys at a time through one
            // short loop, in place in tensor memory, before the rest: few units, and each instruction of an item's
            // code that is fetched anew takes 5 cycles.
            bool slow = masked;
            if constexpr (kDistance) slow = slow || __any_sync(0xFFFFFFFFu, key0 + 127 > my_pos);
            if constexpr (kCapped) {                         // (and those with a score that is many caps)
              if (!slow) {
                load();
                top = top_of();
                slow = __any_sync(0xFFFFFFFFu, top > 0.5f * most);
              }
            }
            if (slow) {
              const Row vis = Row(p, w.s, w.row0 + min(my_row, rows - 1), doc);
              const int first_key = kDistance ? key0 : w.span.key0(u);
#pragma unroll 1
              for (int i = 0; i < 4; ++i) {
                uint32_t x[32];
                const int at = first_key + 32 * i;
                const uint32_t seen = seen_of(vis, at);
                if ((kCapped || kDistance) && __all_sync(0xFFFFFFFFu, seen == 0)) {
#pragma unroll
                  for (int e = 0; e < 32; ++e) x[e] = __float_as_uint(kNegInf);
                  tmem_st32(s_tmem + 32 * i, x);
                  continue;
                }
                tmem_ld32(s_tmem + 32 * i, x);
                tmem_ld_wait();
                hide(seen, x);
                if constexpr (kCapped) {
#pragma unroll
                  for (int e = 0; e < 32; ++e) x[e] = __float_as_uint(min_nan(__uint_as_float(x[e]), most));
#pragma unroll
                  for (int e = 0; e < 32; e += 4) cap4(&x[e], p.cap_in);
                }
                if constexpr (kDistance) {
                  const float base = static_cast<float>(at - my_pos);
#pragma unroll
                  for (int e = 0; e < 32; ++e)
                    x[e] = __float_as_uint(fmaf(__uint_as_float(x[e]), cap_scale, -slope * fabsf(base + e)));
                }
                if constexpr (kCapped) hide(seen, x);     // (what was hidden before came out as -1)
                tmem_st32(s_tmem + 32 * i, x);
              }
              tmem_st_wait();
            }
            if (!kCapped || slow) load();
            if constexpr (kForm == Form::kCappedDistance) {
              if (!slow) cap128(s, p.cap_in);
            }
            if constexpr (kDistance) {
              if (!slow) {                                   // left of the row's place the bias grows evenly with the key
                // From the nearest of 32 keys outwards: each sum is then off by 2^-24 of at most its own key's bias, where sums that
                // began at the far end would carry that end's roundings to keys whose bias is next to nothing.
                const uint64_t scale2 = pair(cap_scale, cap_scale), step2 = pair(-4.f * slope, -4.f * slope);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                  const float base = static_cast<float>(key0 - my_pos + 32 * i + 28);
                  uint64_t bias2[2] = {pair(slope * base, slope * (base + 1.f)), pair(slope * (base + 2.f), slope * (base + 3.f))};
#pragma unroll
                  for (int e = 30; e >= 0; e -= 2) {
                    uint64_t& b = bias2[e >> 1 & 1];
                    const float2 x = unpair(fma2(pair(__uint_as_float(s[i][e]), __uint_as_float(s[i][e + 1])), scale2, b));
                    s[i][e] = __float_as_uint(x.x), s[i][e + 1] = __float_as_uint(x.y);
                    if (e >= 4) b = add2(b, step2);
                  }
                }
              }
            }
            if constexpr (kForm == Form::kCapped) {
              if (!slow) {                                   // (the largest result is that of the largest score)
                top = -rcp_fast(1.f + exp2_fast(top * p.cap_in));   // (of an infinite one, too)
                cap128(s, p.cap_in);
              } else {
                top = top_of();
              }
            } else {
              top = top_of();
            }
          }
          // (the first finite maximum after none needs no rescaling: O and l are zero)
          const bool renew = top > m && (m == kNegInf || (top - m) * scale > kLazy);
          if (__any_sync(0xFFFFFFFFu, renew)) {
            if (__any_sync(0xFFFFFFFFu, renew && m != kNegInf)) {
              const float f = !renew ? 1.f : m == kNegInf ? 0.f : exp2_fast(addend(top) - addend(m));
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
          const float add = addend(m);
          const uint64_t scale2 = pair(scale, scale), addend2 = pair(add, add);
          uint64_t sum2[2] = {};
          auto give = [&](int of) {                        // 64 keys of P are complete
            tmem_st_wait();
            tc_fence_before();
            __syncwarp();
            if (lane == 0 && ok) mbar_arrive(&ctl.p_full[half][of]);
          };
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            uint32_t packed[16];
#pragma unroll
            for (int e = 0; e < 32; e += 2) {
              const float2 x = unpair(fma2(pair(__uint_as_float(s[i][e]), __uint_as_float(s[i][e + 1])), scale2, addend2));
              const float a = exp2_fast(x.x), b = exp2_fast(x.y);
              sum2[i & 1] = add2(sum2[i & 1], pair(a, b));
              packed[e >> 1] = Type<T>::pack(a, b);
            }
            tmem_st16(s_tmem + 16 * i, packed);
            if (i & 1) give(i >> 1);
          }
          const float2 sa = unpair(sum2[0]), sb = unpair(sum2[1]);
          l += (sa.x + sa.y) + (sb.x + sb.y);
        }
        if (q_next) send_q();
        look_for_others();
      }

      // Results of this thread's row: O / l and reference + log2 l (nothing seen: zeros, -inf).
      const bool none = l == 0.f;                          // (a NaN score leaves l NaN)
      float lse2 = none ? kNegInf : (kShift - addend(m)) + log2f(l * (1.f / (1 << kShift)));
      if (kCapped) lse2 += p.cap_log2;                         // (left out of every score)
      float mul = none ? 0.f : 1.f / l, mul_other = 0.f;
      const bool paired = mode == Mode::kPair, split = w.split;
      const bool real = mine && my_row < rows;
      const bool tells = real && !(paired && half == 1);   // writes the row's log-sum
      const int col0 = paired ? kDim / 2 * half : 0, col1 = paired ? col0 + kDim / 2 : kDim;
      const int g = w.row0 + min(my_row, rows - 1), t = p.group_div.div(g);
      const long long tok = w.q0 + t;
      const int head = w.h * p.group + g - t * p.group;
      T* to_out = static_cast<T*>(p.out) + tok * p.o_ts + head * p.o_hs;
      // The common case, a whole item. Little is left for after the last product: what
      // runs once an item is bound by the fetching of its code.
      const bool plain = keys && !split;
      if (plain && !paired && real && p.lse) p.lse[tok * p.heads + head] = lse2 * kLn2;
      if (works(mode)) {
        wait(&ctl.o_done[half], o_phase);
        tc_fence_after();
        o_phase ^= 1;
        if (of_half == 1 && lane == 0 && ok) {             // the last unit of this half
          const uint32_t n = unit_count + n_units - 1;
          mbar_arrive(&ctl.v_empty[(paired && ((n_units - 1) & 1) != half ? n - 1 : n) % S::kVStages]);
        }
      }
      if (keys) unit_count += n_units;
      q_sent = q_next;
      // The halves of a pair hold the same rows in the same lanes of tensor memory: they tell
      // each other log-sums and factors, and each joins half the columns of both.
      if (paired) {
        ctl.row_lse[kHalf * half + my_row] = lse2;
        ctl.row_mul[kHalf * half + my_row] = mul;
        tc_fence_before();
      }
      if (split || paired) meet();                         // (and last_one is known)
      if (paired) {
        tc_fence_after();
        const int at = kHalf * (half ^ 1) + my_row;
        const float other = ctl.row_lse[at], top = fmaxf(lse2, other), ref = top == kNegInf ? 0.f : top;
        const float a = exp2_fast(lse2 - ref), b = exp2_fast(other - ref), sum = a + b;
        lse2 = sum == 0.f ? kNegInf : ref + log2f(sum);
        mul = sum == 0.f ? 0.f : mul * a / sum;
        mul_other = sum == 0.f ? 0.f : ctl.row_mul[at] * b / sum;
        if (plain && tells && p.lse) p.lse[tok * p.heads + head] = lse2 * kLn2;
      }
      // 32 columns of this thread's row, normalised
      auto load_o = [&](int c, uint32_t (&o)[32]) {
        __syncwarp();
        tmem_ld32(o_tmem + c, o);
        tmem_ld_wait();
        const uint64_t mul2 = pair(mul, mul);
#pragma unroll
        for (int e = 0; e < 32; e += 2) {
          const float2 x = unpair(fma2(pair(__uint_as_float(o[e]), __uint_as_float(o[e + 1])), mul2, 0));
          o[e] = __float_as_uint(x.x), o[e + 1] = __float_as_uint(x.y);
        }
        if (mul == 0.f) {
#pragma unroll
          for (int e = 0; e < 32; ++e) o[e] = 0;
        }
        if (paired) {
          uint32_t x[32];
          tmem_ld32((half ? o_tmem - kDim : o_tmem + kDim) + c, x);
          tmem_ld_wait();
          if (mul_other != 0.f) {
#pragma unroll
            for (int e = 0; e < 32; ++e)
              o[e] = __float_as_uint(fmaf(__uint_as_float(x[e]), mul_other, __uint_as_float(o[e])));
          }
        }
      };
      auto store_o = [&](int c, const uint32_t (&o)[32]) {
#pragma unroll
        for (int e = 0; e < 32; e += 16) {
          uint32_t v[8];
#pragma unroll
          for (int i = 0; i < 8; ++i)
            v[i] = Type<T>::pack(__uint_as_float(o[e + 2 * i]), __uint_as_float(o[e + 2 * i + 1]));
          if (c + e + 16 <= p.dim) store32(to_out + c + e, v, cp.out32);
          else if (c + e < p.dim) *reinterpret_cast<uint4*>(to_out + c + e) = make_uint4(v[0], v[1], v[2], v[3]);
        }
      };
      if (plain && mine) {
#pragma unroll 1
        for (int c = col0; c < col1; c += 32) {
          uint32_t o[32];
          load_o(c, o);
          if (real) store_o(c, o);
        }
      }
      const int own = static_cast<int>(blockIdx.x), c0 = w.c0, c1 = w.c1;
      auto part_at = [&](int c) { return 2 * c + (c == c0 ? 1 : 0); };     // a CTA's part of an item is its first but where the item begins
      // The last CTA of a split item does not write its part: it joins the others' with
      // its own. A CTA that is the last only once it has written goes round once more.
      bool last = split && ctl.last_one;
      float row_lse = lse2, base = 0.f;                    // of the whole item
      float* to_part = p.part_o + static_cast<long long>(part_at(own)) * kRows * kDim + my_row * 4;
#pragma unroll 1
      while (!plain) {
        if (last && c1 - c0 >= kFewParts) {
          // Many parts, all in memory: a round trip takes 1500 cycles or more, so a thread has the
          // loads of five parts and two pieces of eight columns in flight at a time;
          // neighbouring lanes take neighbouring rows.
          __threadfence();
          if (threadIdx.x == 0) p.counters[c0] = 0;
          const int r = threadIdx.x;
          if (r < rows) {
            float top = kNegInf, sum = 0.f;
#pragma unroll 8
            for (int i = c0; i <= c1; ++i) top = fmaxf(top, __ldcg(p.part_l + part_at(i) * kRows + r));
            const float ref = top == kNegInf ? 0.f : top;
#pragma unroll 8
            for (int i = c0; i <= c1; ++i) sum += exp2_fast(__ldcg(p.part_l + part_at(i) * kRows + r) - ref);
            ctl.row_lse[r] = sum == 0.f ? kNegInf : ref + log2f(sum);
          }
          meet();
          constexpr int kThreads8 = 32 * kSoftmaxWarps, kBatch = 2, kGroup = 5;
          const int work = rows * (kDim / 8);
#pragma unroll 1
          for (int i0 = threadIdx.x; i0 < work; i0 += kBatch * kThreads8) {
            float x[kBatch][8], from0[kBatch];
            int row[kBatch], col[kBatch];
#pragma unroll
            for (int b = 0; b < kBatch; ++b) {
              const int at = min(i0 + b * kThreads8, work - 1);
              col[b] = at / rows;
              row[b] = at - col[b] * rows;
              from0[b] = ctl.row_lse[row[b]] == kNegInf ? 0.f : ctl.row_lse[row[b]];
#pragma unroll
              for (int e = 0; e < 8; ++e) x[b][e] = 0.f;
            }
#pragma unroll 1
            for (int i = c0; i <= c1; i += kGroup) {
              float4 v[kGroup][kBatch][2];
              float f[kGroup][kBatch];
#pragma unroll
              for (int k = 0; k < kGroup; ++k) {
                const long long from = part_at(min(i + k, c1));
#pragma unroll
                for (int b = 0; b < kBatch; ++b) {
                  f[k][b] = __ldcg(p.part_l + from * kRows + row[b]);
                  const float4* at =
                      reinterpret_cast<const float4*>(p.part_o + (from * kDim + col[b] * 8) * kRows) + row[b];
                  v[k][b][0] = __ldcg(at);
                  v[k][b][1] = __ldcg(at + kRows);
                }
              }
#pragma unroll
              for (int k = 0; k < kGroup; ++k) {
                if (i + k > c1) break;
#pragma unroll
                for (int b = 0; b < kBatch; ++b) {
                  const float g = exp2_fast(f[k][b] - from0[b]);
                  const float4 a = v[k][b][0], c = v[k][b][1];
                  x[b][0] = fmaf(g, a.x, x[b][0]), x[b][1] = fmaf(g, a.y, x[b][1]);
                  x[b][2] = fmaf(g, a.z, x[b][2]), x[b][3] = fmaf(g, a.w, x[b][3]);
                  x[b][4] = fmaf(g, c.x, x[b][4]), x[b][5] = fmaf(g, c.y, x[b][5]);
                  x[b][6] = fmaf(g, c.z, x[b][6]), x[b][7] = fmaf(g, c.w, x[b][7]);
                }
              }
            }
#pragma unroll
            for (int b = 0; b < kBatch; ++b) {
              if (i0 + b * kThreads8 >= work) continue;
              const int gr = w.row0 + row[b], tr = p.group_div.div(gr), hr = w.h * p.group + gr - tr * p.group;
              const long long at = w.q0 + tr;
              if (col[b] * 8 < p.dim)
                *reinterpret_cast<uint4*>(static_cast<T*>(p.out) + at * p.o_ts + hr * p.o_hs + col[b] * 8) =
                    make_uint4(Type<T>::pack(x[b][0], x[b][1]), Type<T>::pack(x[b][2], x[b][3]),
                               Type<T>::pack(x[b][4], x[b][5]), Type<T>::pack(x[b][6], x[b][7]));
              if (p.lse && col[b] == 0) p.lse[at * p.heads + hr] = ctl.row_lse[row[b]] * kLn2;
            }
          }
          break;
        }
        if (last) {
          __threadfence();
          if (threadIdx.x == 0) p.counters[c0] = 0;
          // the log-sum over all parts, in their order; a part then weighs exp2(its own - that)
          float top = lse2, sum = 0.f;
#pragma unroll 1
          for (int pass = 0; pass < 2; ++pass) {
            const float ref = top == kNegInf ? 0.f : top;
#pragma unroll 1
            for (int i = c0; i <= c1; i += 4) {
              float x[4];
#pragma unroll
              for (int k = 0; k < 4; ++k)
                x[k] = i + k > c1 ? kNegInf
                       : i + k == own ? lse2
                                      : __ldcg(p.part_l + part_at(i + k) * kRows + my_row);
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                if (pass == 0) top = fmaxf(top, x[k]);
                else sum += exp2_fast(x[k] - ref);
              }
            }
          }
          const float ref = top == kNegInf ? 0.f : top;
          row_lse = sum == 0.f ? kNegInf : ref + log2f(sum);
          base = sum == 0.f ? 0.f : row_lse;
        }
        if (mine) {
#pragma unroll 1
          for (int c = col0; c < col1; c += 32) {
            uint32_t o[32];
            if (keys) {
              load_o(c, o);
            } else {
#pragma unroll
              for (int e = 0; e < 32; ++e) o[e] = 0;
            }
            if (last) {
              float acc[32];
#pragma unroll
              for (int e = 0; e < 32; ++e) acc[e] = 0.f;
#pragma unroll 1
              for (int i = c0; i <= c1; ++i) {
                if (i == own) {
                  const float f = exp2_fast(lse2 - base);
#pragma unroll
                  for (int e = 0; e < 32; ++e) acc[e] = fmaf(f, __uint_as_float(o[e]), acc[e]);
                } else {
                  const float f = exp2_fast(__ldcg(p.part_l + part_at(i) * kRows + my_row) - base);
                  const float* src = p.part_o + (static_cast<long long>(part_at(i)) * kDim + c) * kRows + my_row * 4;
#pragma unroll
                  for (int e = 0; e < 32; e += 4) {
                    const float4 x = __ldcg(reinterpret_cast<const float4*>(src + e * kRows));
                    acc[e] = fmaf(f, x.x, acc[e]);
                    acc[e + 1] = fmaf(f, x.y, acc[e + 1]);
                    acc[e + 2] = fmaf(f, x.z, acc[e + 2]);
                    acc[e + 3] = fmaf(f, x.w, acc[e + 3]);
                  }
                }
              }
#pragma unroll
              for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(acc[e]);
            }
            if (real && split && !last) {
#pragma unroll
              for (int e = 0; e < 32; e += 4)
                *reinterpret_cast<uint4*>(to_part + (c + e) * kRows) = make_uint4(o[e], o[e + 1], o[e + 2], o[e + 3]);
            } else if (real) {
              store_o(c, o);
            }
          }
          if (tells && split && !last) p.part_l[part_at(own) * kRows + my_row] = lse2;
          else if (tells && p.lse) p.lse[tok * p.heads + head] = row_lse * kLn2;
        }
        if (!split || last) break;
        meet();
        if (threadIdx.x == 0) {
          __threadfence();                                 // covers what the others wrote before they met
          ctl.last_one = atomicAdd(p.counters + c0, 1u) == static_cast<unsigned>(c1 - c0);
        }
        meet();
        last = ctl.last_one;
        if (!last) break;
      }
      tc_fence_before();
      if (paired || split) meet();                         // all of it has been read
      job_done(k);
    }
    all_out();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == kMmaWarp) tmem_dealloc(tmem, 512);
}

// The driver's tensor-map encoder, resolved once through the runtime.
PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encoder() {
  static const PFN_cuTensorMapEncodeTiled_v12000 fn = [] {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult found;
    const bool ok = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &found) ==
                        cudaSuccess && found == cudaDriverEntryPointSuccess;
    return ok ? reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(f) : nullptr;
  }();
  return fn;
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
  const PFN_cuTensorMapEncodeTiled_v12000 encode = tensor_map_encoder();
  if (!encode) return cudaErrorNotSupported;
  const uint32_t steps[4] = {1, 1, 1, 1};
  const CUresult r = encode(map, t == FloatType::BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16,
                            4, const_cast<void*>(base), dims, strides, box, steps, CU_TENSOR_MAP_INTERLEAVE_NONE,
                            CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

template <typename T, int kDim, Form kForm, bool kLimited = false>
cudaError_t launch(const CUtensorMap& km, const CUtensorMap& vm, const ChunkParams& cp, int ctas, cudaStream_t stream) {
  constexpr int kBytes = kSmem<kDim, kForm != Form::kPlain>;
  const cudaError_t e =
      ensure_smem_limit(reinterpret_cast<const void*>(paged_chunk_kernel<T, kDim, kForm, kLimited>), kBytes);
  if (e != cudaSuccess) return e;
  return launch_dependent(paged_chunk_kernel<T, kDim, kForm, kLimited>, ctas, kThreads, kBytes, stream, km, vm, cp);
}

template <Form kForm>
cudaError_t launch_chunk(FloatType t, const PagedParams& params, void* workspace, int num_sms, cudaStream_t stream,
                         unsigned long long wait_ns) {
  ChunkParams cp{};
  cp.p = params;
  cp.wait_ns = wait_ns;
  PagedParams& p = cp.p;
  const int ctas = std::min(num_sms, static_cast<int>(kPagedCounterBytes / sizeof(unsigned)));
  p.counters = static_cast<unsigned*>(workspace);
  // 32-byte stores: the workspace itself is only 16-byte aligned
  p.part_o = reinterpret_cast<float*>((reinterpret_cast<uintptr_t>(workspace) + kPagedCounterBytes + 31) & ~31ull);
  cp.out32 = reinterpret_cast<uintptr_t>(p.out) % 32 == 0 && (p.tokens == 1 || p.o_ts % 16 == 0) &&
             (p.heads == 1 || p.o_hs % 16 == 0);
  const size_t dim = p.dim <= 64 ? 64 : 128;
  p.part_l = p.part_o + 2 * ctas * kRows * dim;
  CUtensorMap km, vm;
  cudaError_t e = encode_cache(&km, &cp.k_heads_first, p.kc, t, p, p.k_ps, p.k_ss, p.k_hs);
  if (e == cudaSuccess) e = encode_cache(&vm, &cp.v_heads_first, p.vc, t, p, p.v_ps, p.v_ss, p.v_hs);
  if (e != cudaSuccess) return e;
  if constexpr (kForm == Form::kPlain) {
    if (wait_ns != kOwnWaitLimit)
      return paged_chunk_limit_ok(t, p.dim) ? launch<__half, 128, Form::kPlain, true>(km, vm, cp, ctas, stream)
                                            : cudaErrorNotSupported;
  }
  if (t == FloatType::BF16)
    return p.dim <= 64 ? launch<__nv_bfloat16, 64, kForm>(km, vm, cp, ctas, stream)
                       : launch<__nv_bfloat16, 128, kForm>(km, vm, cp, ctas, stream);
  return p.dim <= 64 ? launch<__half, 64, kForm>(km, vm, cp, ctas, stream)
                     : launch<__half, 128, kForm>(km, vm, cp, ctas, stream);
}

unsigned read_and_clear_errors() {
  unsigned v = 0;
  if (cudaMemcpyFromSymbol(&v, g_chunk_err, sizeof(v)) != cudaSuccess) return 0xFFFFFFFFu;
  const unsigned zero = 0;
  cudaMemcpyToSymbol(g_chunk_err, &zero, sizeof(zero));
  return v;
}

}  // namespace
}  // namespace kaio
