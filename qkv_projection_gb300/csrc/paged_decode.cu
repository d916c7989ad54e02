// Attention of few rows over a paged cache: single tokens, or any number of
// rows at less than the tensor cores' rate. The general rule of the visible
// keys, the line of work and the joining of split items are in
// paged_attention.cuh.
//
// Online softmax: for each row a running maximum m and sum l over the keys seen
// so far, and the output scaled by exp2(-m); a new maximum rescales l and the
// output. Scores, statistics and outputs are f32; the weights are rounded to the
// tensors' 16-bit type as the operand of the second product (relative error
// 2^-11 or 2^-8 each, the same as the rounding of the result).
//
// What bounds it: the bytes of K and V, each read once. Every warp streams its
// own 16 keys of a 64-key unit through its own ring of shared-memory stages with
// 16-byte asynchronous copies and computes with warp-level m16n8k16 products
// (up to 16 rows; the rate does not matter here, the rows are few), so the main
// loop has no barrier between warps. Keys that no row of the item sees are
// filled with zeros and their pages are not read.
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
constexpr int kMinUnits = 2;                     // units worth a CTA of their own
constexpr int kWhole = 0;                        // units of an item that is not split
using Walk = PagedWalk<kRows, kUnitKeys, kPagedMaxLen, kWhole>;    // (no heavy items)
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
  static __device__ __forceinline__ void run(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    mma_16816(d, a, b0, b1);
  }
  static __device__ __forceinline__ uint32_t pack(float lo, float hi) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
};
template <> struct Mma<__nv_bfloat16> {
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

template <typename T, int kDim>
__global__ void __launch_bounds__(kThreads, kCtasPerSm) paged_decode_kernel(const __grid_constant__ PagedParams p) {
  using S = Shape<kDim>;
  extern __shared__ __align__(128) unsigned char smem[];
  __shared__ long long sums[kThreads];
  __shared__ Walk place;
  __shared__ float warp_m[kWarps][kRows], warp_l[kWarps][kRows];
  __shared__ int last_one;

  allow_dependents_launch();
  grid_dependency_wait();
  PagedShare share;
  if (!paged_share<kThreads>(p, blockIdx.x, gridDim.x, kMinUnits, sums, &place, &share)) return;
  Walk w = place;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  unsigned char* ring = smem + warp * S::kStages * S::kStage;
  const uint32_t ring_addr = smem_u32(ring);
  const int page_mask = (1 << p.page_shift) - 1;

  // this lane's place in a step's copies: one chunk of every (32 / kChunks)-th key
  const int chunk = lane % S::kChunks, key_in_step = lane / S::kChunks;
  constexpr int kKeyStep = 32 / S::kChunks;
  const bool chunk_real = chunk * 8 < p.dim;
  // this lane's rows of the score tile
  const int row_a = lane >> 2, row_b = row_a + 8;

  for (;;) {
    const Span span(p, w.s, w.row0(), w.row1(p));
    const int rows = w.row1(p) - w.row0();
    const int u0 = w.unit, u1 = w.unit_at(p, share.end);
    if (u1 <= u0) break;
    const int steps = span.hi > 0 ? u1 - u0 : 0;
    const T* kbase = static_cast<const T*>(p.kc) + w.h * p.k_hs + chunk * 8;
    const T* vbase = static_cast<const T*>(p.vc) + w.h * p.v_hs + chunk * 8;

    // Q fragments (A operand): rows past the item's are zero
    uint32_t qf[kDim / 16][4];
    {
      const int ra = min(row_a, rows - 1), rb = min(row_b, rows - 1);
      const int ta = (w.row0() + ra) / p.group, tb = (w.row0() + rb) / p.group;
      const int ha = w.h * p.group + (w.row0() + ra) % p.group, hb = w.h * p.group + (w.row0() + rb) % p.group;
      const T* qa = static_cast<const T*>(p.q) + (w.s.q0 + ta) * p.q_ts + ha * p.q_hs;
      const T* qb = static_cast<const T*>(p.q) + (w.s.q0 + tb) * p.q_ts + hb * p.q_hs;
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
    const PagedRow vis_a(p, w.s, w.row0() + min(row_a, rows - 1)), vis_b(p, w.s, w.row0() + min(row_b, rows - 1));
    // keys in [all_lo, all_hi) are seen by every row
    const int all_hi = PagedRow(p, w.s, w.row0()).hi, all_lo = PagedRow(p, w.s, w.row1(p) - 1).lo;

    float o[kDim / 8][4];
#pragma unroll
    for (int n = 0; n < kDim / 8; ++n) o[n][0] = o[n][1] = o[n][2] = o[n][3] = 0.f;
    float m_a = kNegInf, m_b = kNegInf, l_a = 0.f, l_b = 0.f;

    // Page ids of 32 steps at a time, one a lane; the next 32 are fetched while these are used.
    const int* table = p.table + w.b * p.table_stride;
    auto page_of = [&](int step) {
      int id = -1;
      if (step < steps) {
        const int k0 = span.key0(u0 + step) + warp * kStepKeys;
        const bool seen = k0 < span.hi && (k0 + kStepKeys > span.lo || k0 < span.first);
        if (seen) id = table[k0 >> p.page_shift];
        if (id >= p.num_pages) id = -1;
      }
      return id;
    };
    int ids = page_of(lane), ids_next = page_of(32 + lane);

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
          const bool real = id >= 0 && chunk_real && j < span.hi && (j >= span.lo || j < span.first);
          const int at = key * S::kRowBytes + ((chunk ^ (key & 7)) << 4);
          cp_async16(st + at, real ? kp + key * p.k_ss : static_cast<const T*>(p.kc), real ? 16 : 0);
          cp_async16(st + S::kTile + at, real ? vp + key * p.v_ss : static_cast<const T*>(p.vc), real ? 16 : 0);
        }
      }
      cp_async_commit();
    };

#pragma unroll 1
    for (int i = 0; i < S::kStages - 1; ++i) issue(i);
#pragma unroll 1
    for (int step = 0; step < steps; ++step) {
      cp_async_wait<S::kStages - 2>();
      __syncwarp();
      issue(step + S::kStages - 1);
      const uint32_t st = ring_addr + (step % S::kStages) * S::kStage;
      const int k0 = span.key0(u0 + step) + warp * kStepKeys;
      if (k0 >= span.hi) continue;      // this warp's keys of the last unit lie past the end

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
      const float ref_a = top_a == kNegInf ? 0.f : top_a, ref_b = top_b == kNegInf ? 0.f : top_b;
      if (__any_sync(0xFFFFFFFFu, top_a != m_a || top_b != m_b)) {
        const float fa = exp2_fast(m_a - ref_a), fb = exp2_fast(m_b - ref_b);
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

    // The four warps' results are joined through shared memory (the ring's first stages).
    l_a = quad_sum(l_a);
    l_b = quad_sum(l_b);
    float* mine = reinterpret_cast<float*>(ring);
    if ((lane & 3) == 0) {
      warp_m[warp][row_a] = m_a;
      warp_m[warp][row_b] = m_b;
      warp_l[warp][row_a] = l_a;
      warp_l[warp][row_b] = l_b;
    }
#pragma unroll
    for (int n = 0; n < kDim / 8; ++n) {
      const int c = 8 * n + 2 * (lane & 3);
      *reinterpret_cast<float2*>(mine + row_a * kDim + c) = make_float2(o[n][0], o[n][1]);
      *reinterpret_cast<float2*>(mine + row_b * kDim + c) = make_float2(o[n][2], o[n][3]);
    }
    __syncthreads();

    // thread: one row, kSeg columns
    constexpr int kSeg = kRows * kDim / kThreads;
    const int row = threadIdx.x / (kThreads / kRows), col = threadIdx.x % (kThreads / kRows) * kSeg;
    const bool whole_item = u0 == 0 && u1 == w.units;
    const int tok = w.s.q0 + (w.row0() + row) / p.group, head = w.h * p.group + (w.row0() + row) % p.group;
    float acc[kSeg];
    float lse2 = kNegInf;
    if (row < rows) {
      float top = kNegInf, sum = 0.f, f[kWarps];
#pragma unroll
      for (int i = 0; i < kWarps; ++i) top = fmaxf(top, warp_m[i][row]);
      const float ref = top == kNegInf ? 0.f : top;
#pragma unroll
      for (int i = 0; i < kWarps; ++i) {
        f[i] = exp2_fast(warp_m[i][row] - ref);
        sum += f[i] * warp_l[i][row];
      }
      // the sum is zero exactly when nothing was seen: zeros, and a log-sum of -inf
      // (a NaN score leaves a NaN sum)
      lse2 = sum == 0.f ? kNegInf : ref + log2f(sum);
      const float inv = sum == 0.f ? 0.f : 1.f / sum;
#pragma unroll
      for (int c = 0; c < kSeg; ++c) acc[c] = 0.f;
#pragma unroll
      for (int i = 0; i < kWarps; ++i) {
        const float* src = reinterpret_cast<const float*>(smem + i * S::kStages * S::kStage) + row * kDim + col;
#pragma unroll
        for (int c = 0; c < kSeg; c += 4) {
          const float4 v = *reinterpret_cast<const float4*>(src + c);
          acc[c] += f[i] * v.x;
          acc[c + 1] += f[i] * v.y;
          acc[c + 2] += f[i] * v.z;
          acc[c + 3] += f[i] * v.w;
        }
      }
#pragma unroll
      for (int c = 0; c < kSeg; ++c) acc[c] *= inv;
    }

    bool write = whole_item;
    if (!whole_item) {
      const int slot = 2 * static_cast<int>(blockIdx.x) + (u0 == 0 ? 1 : 0);
      if (row < rows) {
        float* dst = p.part_o + (static_cast<long long>(slot) * kRows + row) * kDim + col;
#pragma unroll
        for (int c = 0; c < kSeg; c += 4)
          *reinterpret_cast<float4*>(dst + c) = make_float4(acc[c], acc[c + 1], acc[c + 2], acc[c + 3]);
        if (col == 0) p.part_l[slot * kRows + row] = lse2;
      }
      const int c0 = share.owner(w.place_of(p, 0)), c1 = share.owner(w.place_of(p, w.units - 1));
      __threadfence();
      __syncthreads();
      if (threadIdx.x == 0) {
        const unsigned seen = atomicAdd(p.counters + c0, 1u);
        last_one = seen == static_cast<unsigned>(c1 - c0);
        if (last_one) p.counters[c0] = 0;
      }
      __syncthreads();
      if (last_one) {
        // Few rows leave most threads without one: then 2, 4, 8 or 16 groups of
        // threads take every 2nd, 4th, ... part, and are added up in shared memory.
        __threadfence();
        write = true;
        int groups = kRows;
        while (groups * rows > kRows) groups >>= 1;
        const int group = row / (kRows / groups), r = row % (kRows / groups);
        float top = kNegInf, sum = 0.f;
#pragma unroll
        for (int c = 0; c < kSeg; ++c) acc[c] = 0.f;
        if (r < rows) {
#pragma unroll 4
          for (int c = c0; c <= c1; ++c)
            top = fmaxf(top, __ldcg(p.part_l + (2 * c + (c == c0 ? 1 : 0)) * kRows + r));
        }
        const float ref = top == kNegInf ? 0.f : top;
        if (r < rows) {
#pragma unroll 4
          for (int c = c0 + group; c <= c1; c += groups) {
            const int from = 2 * c + (c == c0 ? 1 : 0);
            const float f = exp2_fast(__ldcg(p.part_l + from * kRows + r) - ref);
            sum += f;
            const float* src = p.part_o + (static_cast<long long>(from) * kRows + r) * kDim + col;
#pragma unroll
            for (int e = 0; e < kSeg; e += 4) {
              const float4 v = __ldcg(reinterpret_cast<const float4*>(src + e));
              acc[e] += f * v.x;
              acc[e + 1] += f * v.y;
              acc[e + 2] += f * v.z;
              acc[e + 3] += f * v.w;
            }
          }
        }
        if (groups > 1) {
          float* joined = reinterpret_cast<float*>(smem);     // [kRows][kDim], and the sums after it
#pragma unroll
          for (int c = 0; c < kSeg; c += 4)
            *reinterpret_cast<float4*>(joined + row * kDim + col + c) =
                make_float4(acc[c], acc[c + 1], acc[c + 2], acc[c + 3]);
          if (col == 0) joined[kRows * kDim + row] = sum;
          __syncthreads();
          if (row < rows) {
            for (int g = 1; g < groups; ++g) {
              const int other = row + g * (kRows / groups);
              sum += joined[kRows * kDim + other];
#pragma unroll
              for (int c = 0; c < kSeg; c += 4) {
                const float4 v = *reinterpret_cast<const float4*>(joined + other * kDim + col + c);
                acc[c] += v.x, acc[c + 1] += v.y, acc[c + 2] += v.z, acc[c + 3] += v.w;
              }
            }
          }
        }
        lse2 = sum == 0.f ? kNegInf : ref + log2f(sum);
        const float inv = sum == 0.f ? 0.f : 1.f / sum;
#pragma unroll
        for (int c = 0; c < kSeg; ++c) acc[c] *= inv;
      }
    }
    if (write && row < rows) {
      T* dst = static_cast<T*>(p.out) + tok * p.o_ts + head * p.o_hs + col;
#pragma unroll
      for (int c = 0; c < kSeg; c += 8) {
        if (col + c < p.dim) {
          uint4 v;
          v.x = Mma<T>::pack(acc[c], acc[c + 1]);
          v.y = Mma<T>::pack(acc[c + 2], acc[c + 3]);
          v.z = Mma<T>::pack(acc[c + 4], acc[c + 5]);
          v.w = Mma<T>::pack(acc[c + 6], acc[c + 7]);
          *reinterpret_cast<uint4*>(dst + c) = v;
        }
      }
      if (p.lse && col == 0) p.lse[static_cast<long long>(tok) * p.heads + head] = lse2 * kLn2;
    }
    __syncthreads();       // shared memory is free for the next item
    if (u1 < w.units) break;
    w.next_item(p);
    if (w.b >= p.batch) break;
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
  // No more CTAs than counters, and than there can be shares of kMinUnits units.
  const long long most = static_cast<long long>(p.max_pages) << p.page_shift;
  const long long units = (most + kUnitKeys - 1) / kUnitKeys + 1;
  const long long tiles = (static_cast<long long>(p.tokens) * p.group + kRows - 1) / kRows + p.batch;
  int ctas = std::min(num_sms * kCtasPerSm, static_cast<int>(kPagedCounterBytes / sizeof(unsigned)));
  ctas = static_cast<int>(std::max(1ll, std::min<long long>(ctas, units * tiles * p.kv_heads / kMinUnits)));
  p.counters = static_cast<unsigned*>(workspace);
  p.part_o = reinterpret_cast<float*>(static_cast<char*>(workspace) + kPagedCounterBytes);
  p.part_l = p.part_o + static_cast<size_t>(2) * ctas * kRows * (p.dim <= 64 ? 64 : 128);
  if (t == FloatType::BF16)
    return p.dim <= 64 ? launch<__nv_bfloat16, 64>(p, ctas, stream) : launch<__nv_bfloat16, 128>(p, ctas, stream);
  return p.dim <= 64 ? launch<__half, 64>(p, ctas, stream) : launch<__half, 128>(p, ctas, stream);
}

}  // namespace kaio
