// Attention of few rows over a paged cache: single tokens, or any number of
// rows at less than the tensor cores' rate. The general rule of the visible
// keys, the line of work and the joining of split items are in
// paged_attention.cuh.
//
// Online softmax: for each row a running maximum m and sum l over the keys seen
// so far, and the output scaled by exp2(-m); a new maximum rescales l and the
// output. Scores, statistics and outputs are f32; the weights are rounded to the
// tensors' 16-bit type as the operand of the second product. That is a relative error of
// 2^-8 each in bf16, the same as the rounding of the result. An f16 holds 2^-11 only down
// to 2^-14 and nothing below 2^-25, and many keys far below one may weigh as much
// together as they are many, so its weights are exp2(s - m + 14): the largest is 2^14 of
// the 65504 that fit, and what is lost lies 2^-39 below it.
//
// What bounds it: the bytes of K and V, each read once. Every warp streams its
// own 16 keys of a 64-key unit through its own ring of shared-memory stages with
// 16-byte asynchronous copies and computes with warp-level m16n8k16 products
// (up to 16 rows; the rate does not matter here, the rows are few), so the main
// loop has no barrier between warps. Keys that no row of the item sees are
// filled with zeros and their pages are not read. Two CTAs of four warps on an SM
// with three or six stages of 8 or 4 KB each keep 150 to 190 KB in flight on it.
// 64 tokens over contexts of up to 8192, 32 heads on 8 of 128: 203-210 us, 6.4-6.7 TB/s
// (0.95-0.98 of a measured copy); one token over 131071: 90-91 us (0.87); 16 tokens of 64
// heads with a window of 4096: 52-54 us (0.75; 5 us of it before the first keys arrive).
//
// Short calls are bound by what surrounds the units. One token over 1037 keys, 32 heads
// (12.0 us): 4 us from the launch to the first copies (the shares, then page ids, then
// keys: three round trips, in code that is fetched for the first time), 2 us for two
// units, 4 us to write a part, to find out who is last and to join nine of them.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>
#include <cstdint>

#include "paged_attention.cuh"

namespace kaio {
namespace {

constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;
constexpr int kStepKeys = 16;                    // keys of one warp and step
constexpr int kUnitKeys = kWarps * kStepKeys;    // 64
constexpr int kRows = kPagedDecodeRows;
constexpr int kCtasPerSm = 2;
// Joining parts takes 4-6 us, a unit 0.6 us (32 sequences of 300 positions, 5 units: 10.0 us
// whole, 16.5 us split; 64 of 900, 15 units to shares of 13: 20.6 whole, 25.3 split). A part is
// worth 0.2 units in the size of shares (one token over 9000 keys, 32/8 heads: 17.1 us, with 0.4
// 18.4, 0.8 22.6; 4 over 2000: 13.6, 13.3, 15.0).
struct Work {
  static constexpr int kRows = kPagedDecodeRows, kFewRows = kRows, kKeys = kUnitKeys;
  static constexpr int kCost = 4, kSmallRows = 0, kSmallCost = 4, kItemCost = 8, kSnap = 12;
  static constexpr int kWhole = 8, kJoin = 8, kWholeOfMany = 8;
  static constexpr float kPartWorth = 0.2f;
};
using Walk = PagedWalk<Work>;
using Span = PagedSpan<kUnitKeys>;

template <int kDim> struct Shape {
  static constexpr int kRowBytes = kDim * 2;
  static constexpr int kTile = kStepKeys * kRowBytes;     // K or V of one step
  static constexpr int kStage = 2 * kTile;
  static constexpr int kStages = kDim == 128 ? 3 : 6;
  static constexpr int kSmem = kWarps * kStages * kStage;
  static constexpr int kChunks = kDim / 8;                // 16-byte chunks of a row
};

template <typename T> struct Mma;
template <> struct Mma<__half> {
  static constexpr int kShift = 14;      // log2 of the largest weight
  static __device__ __forceinline__ void run(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    mma_16816(d, a, b0, b1);
  }
  static __device__ __forceinline__ uint32_t pack(float lo, float hi) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
};
template <> struct Mma<__nv_bfloat16> {
  static constexpr int kShift = 0;       // (f32's range)
  static __device__ __forceinline__ void run(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  }
  static __device__ __forceinline__ uint32_t pack(float lo, float hi) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
};

__device__ __forceinline__ void ldmatrix4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldmatrix4_trans(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int kPending> __device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(kPending) : "memory");
}

__device__ __forceinline__ float quad_max(float v) {
  v = fmaxf(v, __shfl_xor_sync(0xFFFFFFFFu, v, 1));
  return fmaxf(v, __shfl_xor_sync(0xFFFFFFFFu, v, 2));
}
__device__ __forceinline__ float quad_sum(float v) {
  v += __shfl_xor_sync(0xFFFFFFFFu, v, 1);
  return v + __shfl_xor_sync(0xFFFFFFFFu, v, 2);
}

// What the exponents of a row with maximum m are relative to. Rounded up, so that at any
// size of m the largest weight is between 1 and 2^kShift.
template <int kShift> __device__ __forceinline__ float reference(float m) {
  return kShift ? __fadd_ru(m, -static_cast<float>(kShift)) : m;
}

// Shared memory of a CTA: a ring for each warp. Between items the first stage
// already takes the next item's first keys; the others hold what the warps and CTAs
// tell each other (kScratch floats of each warp's are used as one array).
template <typename T, int kDim>
__global__ void __launch_bounds__(kThreads, kCtasPerSm) paged_decode_kernel(const __grid_constant__ PagedParams p) {
  using S = Shape<kDim>;
  constexpr int kShift = Mma<T>::kShift;
  extern __shared__ __align__(128) unsigned char smem[];
  __shared__ long long sums[2 * kWarps];
  __shared__ Walk place;
  __shared__ float warp_ref[kWarps][kRows], warp_l[kWarps][kRows], own_lse[kRows];
  __shared__ int last_one;

  allow_dependents_launch();
  grid_dependency_wait();
  PagedShare share;
  if (!paged_share<kThreads>(p, blockIdx.x, gridDim.x, sums, &place, &share)) return;
  Walk w = place;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  constexpr int kRing = S::kStages * S::kStage;
  unsigned char* ring = smem + warp * kRing;
  const uint32_t ring_addr = smem_u32(ring);
  const int page_mask = (1 << p.page_shift) - 1;
  // rows of the warps' outputs are padded by eight floats: four rows' stores then fall on different banks
  constexpr int kPad = kDim + 8;
  auto scratch = [&](int of_warp) { return reinterpret_cast<float*>(smem + of_warp * kRing + S::kStage); };
  constexpr int kScratch = 4096;
  static_assert(kScratch * 4 <= kRing - S::kStage && kRows * kPad <= kScratch, "scratch");
  auto weight_at = [&](int i) { return scratch(i / kScratch) + i % kScratch; };

  // this lane's place in a step's copies: one chunk of every (32 / kChunks)-th key
  const int chunk = lane % S::kChunks, key_in_step = lane / S::kChunks;
  constexpr int kKeyStep = 32 / S::kChunks;
  const bool chunk_real = chunk * 8 < p.dim;
  // this lane's rows of the score tile
  const int row_a = lane >> 2, row_b = row_a + 8;

  // What the copies of the item at `w` go by.
  int lo, hi, first, u0, u1, steps, ids, ids_next;
  Span span(p, w.s, w.row0(), w.row1(p));
  const T *kbase, *vbase;
  const int* table;
  // Page ids of 32 steps at a time, one a lane; the next 32 are fetched while these are used.
  auto page_of = [&](int step) {
    int id = -1;
    if (step < steps) {
      const int k0 = span.key0(u0 + step) + warp * kStepKeys;
      const bool seen = k0 < hi && (k0 + kStepKeys > lo || k0 < first);
      if (seen) id = table[k0 >> p.page_shift];
      if (id >= p.num_pages) id = -1;
    }
    return id;
  };
  auto issue = [&](int step) {
    if (step < steps) {
      if (step > 0 && (step & 31) == 0) {
        ids = ids_next;
        ids_next = page_of(step + 32 + lane);
      }
      const int id = __shfl_sync(0xFFFFFFFFu, ids, step & 31);
      const int k0 = span.key0(u0 + step) + warp * kStepKeys;
      const long long slot0 = k0 & page_mask;
      const T* kp = kbase + (id < 0 ? 0 : id * p.k_ps + slot0 * p.k_ss);
      const T* vp = vbase + (id < 0 ? 0 : id * p.v_ps + slot0 * p.v_ss);
      unsigned char* st = ring + (step % S::kStages) * S::kStage;
#pragma unroll
      for (int i = 0; i < kStepKeys / kKeyStep; ++i) {
        const int key = key_in_step + i * kKeyStep;
        const int j = k0 + key;
        const bool real = id >= 0 && chunk_real && j < hi && (j >= lo || j < first);
        const int at = key * S::kRowBytes + ((chunk ^ (key & 7)) << 4);
        cp_async16(st + at, real ? kp + key * p.k_ss : static_cast<const T*>(p.kc), real ? 16 : 0);
        cp_async16(st + S::kTile + at, real ? vp + key * p.v_ss : static_cast<const T*>(p.vc), real ? 16 : 0);
      }
    }
    cp_async_commit();
  };
  // Begins the item at `w` (its page ids and first step); false if the share ends before it.
  auto begin = [&] {
    if (w.b >= p.batch) return false;
    u0 = w.unit;
    u1 = w.cut(share.end, share);
    if (u1 <= u0) return false;
    span = Span(p, w.s, w.row0(), w.row1(p));
    lo = span.lo, hi = span.hi, first = span.first;
    steps = hi > 0 ? u1 - u0 : 0;
    kbase = static_cast<const T*>(p.kc) + w.h * p.k_hs + chunk * 8;
    vbase = static_cast<const T*>(p.vc) + w.h * p.v_hs + chunk * 8;
    table = p.table + w.b * p.table_stride;
    ids = page_of(lane);
    ids_next = page_of(32 + lane);
    issue(0);
    return true;
  };
  if (!begin()) return;

#pragma unroll 1
  for (;;) {
    const PagedSeq seq = w.s;
    const int rows = w.row1(p) - w.row0(), row0 = w.row0(), head0 = w.h * p.group;
    const bool split = u0 != 0 || u1 != w.units;
    const int c0 = split ? w.first_owner(share) : 0, c1 = split ? w.last_owner(share) : 0;

    // Q fragments (A operand): rows past the item's are zero
    uint32_t qf[kDim / 16][4];
    {
      const int ra = row0 + min(row_a, rows - 1), rb = row0 + min(row_b, rows - 1);
      const int ta = p.group_div.div(ra), tb = p.group_div.div(rb);
      const T* qa = static_cast<const T*>(p.q) + (seq.q0 + ta) * p.q_ts + (head0 + ra - ta * p.group) * p.q_hs;
      const T* qb = static_cast<const T*>(p.q) + (seq.q0 + tb) * p.q_ts + (head0 + rb - tb * p.group) * p.q_hs;
#pragma unroll
      for (int ks = 0; ks < kDim / 16; ++ks) {
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          const int c = ks * 16 + half * 8 + 2 * (lane & 3);
          const bool in = c < p.dim;
          qf[ks][2 * half] = in && row_a < rows ? *reinterpret_cast<const uint32_t*>(qa + c) : 0u;
          qf[ks][2 * half + 1] = in && row_b < rows ? *reinterpret_cast<const uint32_t*>(qb + c) : 0u;
        }
      }
    }
    const PagedRow vis_a(p, seq, row0 + min(row_a, rows - 1)), vis_b(p, seq, row0 + min(row_b, rows - 1));
    // keys in [all_lo, all_hi) are seen by every row
    const int all_hi = PagedRow(p, seq, row0).hi, all_lo = PagedRow(p, seq, row0 + rows - 1).lo;

    float o[kDim / 8][4];
#pragma unroll
    for (int n = 0; n < kDim / 8; ++n) o[n][0] = o[n][1] = o[n][2] = o[n][3] = 0.f;
    float m_a = kNegInf, m_b = kNegInf, l_a = 0.f, l_b = 0.f;

#pragma unroll 1
    for (int i = 1; i < S::kStages - 1; ++i) issue(i);
#pragma unroll 1
    for (int step = 0; step < steps; ++step) {
      cp_async_wait<S::kStages - 2>();
      __syncwarp();
      issue(step + S::kStages - 1);
      const uint32_t st = ring_addr + (step % S::kStages) * S::kStage;
      const int k0 = span.key0(u0 + step) + warp * kStepKeys;
      if (k0 >= hi) continue;      // this warp's keys of the last unit lie past the end

      // scores of 16 keys: two column tiles of eight
      float s[2][4] = {};
      const int mrow = (lane & 7) + ((lane >> 4) << 3), mcol = (lane >> 3) & 1;
#pragma unroll
      for (int ks = 0; ks < kDim / 16; ++ks) {
        uint32_t kf[4];
        ldmatrix4(st + mrow * S::kRowBytes + (((2 * ks + mcol) ^ (mrow & 7)) << 4), kf);
        Mma<T>::run(s[0], qf[ks], kf[0], kf[1]);
        Mma<T>::run(s[1], qf[ks], kf[2], kf[3]);
      }
      const bool whole = k0 + kStepKeys <= all_hi && (k0 >= all_lo || k0 + kStepKeys <= p.sinks);
#pragma unroll
      for (int n = 0; n < 2; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          s[n][e] *= p.scale_log2;
          if (!whole) {
            const int j = k0 + 8 * n + 2 * (lane & 3) + (e & 1);
            const PagedRow& v = e < 2 ? vis_a : vis_b;
            if (!(j < v.hi && (j >= v.lo || j < p.sinks))) s[n][e] = kNegInf;
          }
        }
      const float top_a = fmaxf(m_a, quad_max(fmaxf(fmaxf(s[0][0], s[0][1]), fmaxf(s[1][0], s[1][1]))));
      const float top_b = fmaxf(m_b, quad_max(fmaxf(fmaxf(s[0][2], s[0][3]), fmaxf(s[1][2], s[1][3]))));
      // a row that has seen nothing yet keeps weights and sums of zero
      const float ref_a = top_a == kNegInf ? 0.f : reference<kShift>(top_a);
      const float ref_b = top_b == kNegInf ? 0.f : reference<kShift>(top_b);
      if (__any_sync(0xFFFFFFFFu, top_a != m_a || top_b != m_b)) {
        const float fa = exp2_fast(reference<kShift>(m_a) - ref_a), fb = exp2_fast(reference<kShift>(m_b) - ref_b);
        l_a *= fa;
        l_b *= fb;
#pragma unroll
        for (int n = 0; n < kDim / 8; ++n) {
          o[n][0] *= fa;
          o[n][1] *= fa;
          o[n][2] *= fb;
          o[n][3] *= fb;
        }
        m_a = top_a;
        m_b = top_b;
      }
#pragma unroll
      for (int n = 0; n < 2; ++n) {
        s[n][0] = exp2_fast(s[n][0] - ref_a);
        s[n][1] = exp2_fast(s[n][1] - ref_a);
        s[n][2] = exp2_fast(s[n][2] - ref_b);
        s[n][3] = exp2_fast(s[n][3] - ref_b);
        l_a += s[n][0] + s[n][1];
        l_b += s[n][2] + s[n][3];
      }
      const uint32_t pf[4] = {Mma<T>::pack(s[0][0], s[0][1]), Mma<T>::pack(s[0][2], s[0][3]),
                              Mma<T>::pack(s[1][0], s[1][1]), Mma<T>::pack(s[1][2], s[1][3])};
      const int vrow = lane & 15, vcol = lane >> 4;
#pragma unroll
      for (int n = 0; n < kDim / 16; ++n) {
        uint32_t vf[4];
        ldmatrix4_trans(st + S::kTile + vrow * S::kRowBytes + (((2 * n + vcol) ^ (vrow & 7)) << 4), vf);
        Mma<T>::run(o[2 * n], pf, vf[0], vf[1]);
        Mma<T>::run(o[2 * n + 1], pf, vf[2], vf[3]);
      }
    }
    cp_async_wait<0>();
    __syncwarp();
    // Of a split item the CTA that finds all other parts written is the last.
    unsigned seen = 0;
    if (split && threadIdx.x == 0)
      asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(seen) : "l"(p.counters + c0) : "memory");

    // The next item's first keys are on their way while this one is finished.
    const bool ends = u1 == w.units;
    bool more = false;
    if (ends) {
      w.next_item(p);
      more = begin();
    }

    // The four warps' results: references, sums and outputs of the real rows.
    l_a = quad_sum(l_a);
    l_b = quad_sum(l_b);
    if ((lane & 3) == 0) {
      warp_ref[warp][row_a] = reference<kShift>(m_a);
      warp_ref[warp][row_b] = reference<kShift>(m_b);
      warp_l[warp][row_a] = l_a;
      warp_l[warp][row_b] = l_b;
    }
    float* mine = scratch(warp);
#pragma unroll
    for (int n = 0; n < kDim / 8; ++n) {
      const int c = 8 * n + 2 * (lane & 3);
      if (row_a < rows) *reinterpret_cast<float2*>(mine + row_a * kPad + c) = make_float2(o[n][0], o[n][1]);
      if (row_b < rows) *reinterpret_cast<float2*>(mine + row_b * kPad + c) = make_float2(o[n][2], o[n][3]);
    }
    if (threadIdx.x == 0) last_one = split && seen == static_cast<unsigned>(c1 - c0);
    __syncthreads();

    // A thread takes four columns of a row at a time; up to kMine of them.
    constexpr int kQuads = kDim / 4, kMine = kRows * kQuads / kThreads;
    const int quads = rows * kQuads;
    float4 acc[kMine];
    float lse2[kMine];
#pragma unroll
    for (int k = 0; k < kMine; ++k) {
      const int i = threadIdx.x + k * kThreads, row = i / kQuads, col = i % kQuads * 4;
      acc[k] = make_float4(0.f, 0.f, 0.f, 0.f);
      lse2[k] = kNegInf;
      if (i >= quads) continue;
      float top = kNegInf, sum = 0.f, f[kWarps];
#pragma unroll
      for (int j = 0; j < kWarps; ++j) top = fmaxf(top, warp_ref[j][row]);
      const float ref = top == kNegInf ? 0.f : top;
#pragma unroll
      for (int j = 0; j < kWarps; ++j) {
        f[j] = exp2_fast(warp_ref[j][row] - ref);
        sum += f[j] * warp_l[j][row];
      }
      // the sum is zero exactly when nothing was seen: zeros, and a log-sum of -inf
      // (a NaN score leaves a NaN sum)
      lse2[k] = sum == 0.f ? kNegInf : (ref + kShift) + log2f(sum * (1.f / (1 << kShift)));
      const float inv = sum == 0.f ? 0.f : 1.f / sum;
#pragma unroll
      for (int j = 0; j < kWarps; ++j) {
        const float4 v = *reinterpret_cast<const float4*>(scratch(j) + row * kPad + col);
        acc[k].x += f[j] * v.x, acc[k].y += f[j] * v.y, acc[k].z += f[j] * v.z, acc[k].w += f[j] * v.w;
      }
      acc[k].x *= inv, acc[k].y *= inv, acc[k].z *= inv, acc[k].w *= inv;
      if (col == 0) own_lse[row] = lse2[k];
    }

    auto part_at = [&](int c) { return 2 * c + (c == c0 ? 1 : 0); };   // a CTA's part of an item is its first but where the item begins
    bool last = split && last_one;
    if (split && !last) {
#pragma unroll
      for (int k = 0; k < kMine; ++k) {
        const int i = threadIdx.x + k * kThreads;
        if (i >= quads) continue;
        *reinterpret_cast<float4*>(p.part_o + static_cast<long long>(part_at(blockIdx.x)) * kRows * kDim + i * 4) = acc[k];
        if (i % kQuads == 0) p.part_l[part_at(blockIdx.x) * kRows + i / kQuads] = lse2[k];
      }
      __syncthreads();
      if (threadIdx.x == 0) {
        __threadfence();                                   // covers what the others wrote before they met
        last_one = atomicAdd(p.counters + c0, 1u) == static_cast<unsigned>(c1 - c0);
      }
      __syncthreads();
      last = last_one;
    }
    if (last) {
      // All parts' log-sums first, then each part weighs exp2(its own - the row's); always in
      // the parts' order. This CTA's own part comes from its registers.
      const int own = static_cast<int>(blockIdx.x), parts = c1 - c0 + 1;
      __threadfence();
      if (threadIdx.x == 0) p.counters[c0] = 0;
      __syncthreads();                                     // the warps' outputs have been read, own_lse is written
#pragma unroll 4
      for (int i = threadIdx.x; i < parts * rows; i += kThreads) {
        const int part = c0 + i / rows, row = i % rows;
        *weight_at(i) = part == own ? own_lse[row] : __ldcg(p.part_l + part_at(part) * kRows + row);
      }
      __syncthreads();
#pragma unroll 1
      for (int i = threadIdx.x; i < rows; i += kThreads) {
        float top = kNegInf, sum = 0.f;
#pragma unroll 8
        for (int c = 0; c < parts; ++c) top = fmaxf(top, *weight_at(c * rows + i));
        const float ref = top == kNegInf ? 0.f : top;
#pragma unroll 8
        for (int c = 0; c < parts; ++c) sum += exp2_fast(*weight_at(c * rows + i) - ref);
        own_lse[i] = sum == 0.f ? kNegInf : ref + log2f(sum);
      }
      __syncthreads();
#pragma unroll
      for (int k = 0; k < kMine; ++k) {
        const int i = threadIdx.x + k * kThreads, row = i / kQuads;
        if (i >= quads) continue;
        const float4 mine4 = acc[k];
        lse2[k] = own_lse[row];
        const float base = lse2[k] == kNegInf ? 0.f : lse2[k];
        acc[k] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
        for (int c = 0; c < parts; ++c) {
          const float f = exp2_fast(*weight_at(c * rows + row) - base);
          const float4 v = c0 + c == own ? mine4
                                         : __ldcg(reinterpret_cast<const float4*>(
                                               p.part_o + static_cast<long long>(part_at(c0 + c)) * kRows * kDim + i * 4));
          acc[k].x += f * v.x, acc[k].y += f * v.y, acc[k].z += f * v.z, acc[k].w += f * v.w;
        }
      }
    }
    if (!split || last) {
#pragma unroll
      for (int k = 0; k < kMine; ++k) {
        const int i = threadIdx.x + k * kThreads, row = row0 + i / kQuads, col = i % kQuads * 4;
        if (i >= quads) continue;
        const int t = p.group_div.div(row);
        const long long tok = seq.q0 + t;
        const int head = head0 + row - t * p.group;
        if (col < p.dim)
          *reinterpret_cast<uint2*>(static_cast<T*>(p.out) + tok * p.o_ts + head * p.o_hs + col) =
              make_uint2(Mma<T>::pack(acc[k].x, acc[k].y), Mma<T>::pack(acc[k].z, acc[k].w));
        if (p.lse && col == 0) p.lse[tok * p.heads + head] = lse2[k] * kLn2;
      }
    }
    if (!more) break;
    __syncthreads();       // the scratch is free for the next item's keys
  }
}

template <typename T, int kDim>
cudaError_t launch(const PagedParams& p, int ctas, cudaStream_t stream) {
  const void* kernel = reinterpret_cast<const void*>(paged_decode_kernel<T, kDim>);
  const cudaError_t e = ensure_smem_limit(kernel, Shape<kDim>::kSmem);
  if (e != cudaSuccess) return e;
  return launch_dependent(paged_decode_kernel<T, kDim>, ctas, kThreads, Shape<kDim>::kSmem, stream, p);
}

}  // namespace

size_t paged_decode_workspace_bytes(int num_sms) {
  const size_t ctas = static_cast<size_t>(num_sms) * kCtasPerSm;
  return kPagedCounterBytes + 2 * ctas * kRows * (128 + 1) * sizeof(float);
}

cudaError_t launch_paged_decode(FloatType t, PagedParams p, void* workspace, int num_sms, cudaStream_t stream) {
  // No more CTAs than counters, and than there can be units.
  const long long most = static_cast<long long>(p.max_pages) << p.page_shift;
  const long long units = (most + kUnitKeys - 1) / kUnitKeys + 1;
  const long long tiles = (static_cast<long long>(p.tokens) * p.group + kRows - 1) / kRows + p.batch;
  int ctas = std::min(num_sms * kCtasPerSm, static_cast<int>(kPagedCounterBytes / sizeof(unsigned)));
  ctas = static_cast<int>(std::max(1ll, std::min<long long>(ctas, units * tiles * p.kv_heads)));
  p.counters = static_cast<unsigned*>(workspace);
  p.part_o = reinterpret_cast<float*>(static_cast<char*>(workspace) + kPagedCounterBytes);
  p.part_l = p.part_o + static_cast<size_t>(2) * ctas * kRows * (p.dim <= 64 ? 64 : 128);
  if (t == FloatType::BF16)
    return p.dim <= 64 ? launch<__nv_bfloat16, 64>(p, ctas, stream) : launch<__nv_bfloat16, 128>(p, ctas, stream);
  return p.dim <= 64 ? launch<__half, 64>(p, ctas, stream) : launch<__half, 128>(p, ctas, stream);
}

}  // namespace kaio
