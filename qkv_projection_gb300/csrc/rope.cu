// Rotary positions with several axes, and the same fused with the write of K
// and V into a paged cache.
//
// Pair i of R pairs belongs to one position axis a(i) (sections of consecutive
// pairs) and turns by angle = pos[a(i), t] * inv_freq[i]:
//   y0 = x0 cos - x1 sin,   y1 = x1 cos + x0 sin     (sin negated: the inverse,
// which is also the gradient, the rotation being orthogonal). Elements past 2R
// are copied. Products and sums in f32, one rounding to the tensors' type.
//
// The angle is reduced in fixed point (the idea of Payne and Hanek, Radian reduction for
// trigonometric functions, 1983): the turns of one position, inv_freq / 2 pi, are held
// modulo one turn in 64 bits, from as many bits of 1 / 2 pi as inv_freq's exponent asks
// for; their product with the integer position wraps modulo one turn by itself, and its
// top 32 bits are the angle in turns. What is dropped before that is 2^-32 turns at any
// position, so the error is that of the angle's f32, 2^-25 turns (an f32 product of
// position and frequency is off by 0.004 radians at position 100000).
//
// What bounds it: with many tokens of many heads, bytes; every value is read once and
// written once, and the sines are computed once per token and pair and shared by all
// heads through shared memory. With fewer, that step: nothing of x is loaded before the
// sines stand there (4099 tokens of 32 heads take 15.2 us for 9.9 of bytes; 3.2 warps wait
// at the barrier for each instruction, and DRAM is at 24 %). A thread moves 32 bytes (both halves of eight pairs) at a time, in few
// registers: eight CTAs of 256 threads on an SM hide the latency better than
// several units in flight per thread (two: 38 us, four: 46 us, one: 37 us for the
// fused write of 8192 tokens of 32 + 8 heads of 128, 5.4 TB/s read and written).
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cstdint>

#include "attention_internal.h"
#include "kaio_device.cuh"

namespace kaio {
namespace {

constexpr int kRopeThreads = 256;
constexpr int kRopeMaxPairs = 128;
constexpr int kRopeMaxTokens = 4;    // tokens of one CTA

struct RopeKernelParams {
  RopeParams r;
  FastDiv unit_div, rot_div, copy_div;   // units per token, per rotated head, per copied head
  int tokens_per_cta;
};

// inv_freq / 2 pi modulo one, in units of 2^-64: with inv_freq = m 2^(e - 150), m of 24 bits,
// it is m times 2^(e - 86) / 2 pi, of which the lowest 64 bits before the point count and 32
// behind it for rounding. (In integers: the same in f64 was a tenth of the gradient's time.)
__device__ __forceinline__ unsigned long long turns_of(float inv_freq) {
  constexpr unsigned __int128 kInv2Pi =      // floor(2^128 / 2 pi)
      static_cast<unsigned __int128>(0x28BE60DB9391054Aull) << 64 | 0x7F09D5F47D4D3770ull;
  const uint32_t bits = __float_as_uint(inv_freq), m = (bits & 0x7FFFFFu) | 0x800000u;
  const int right = 182 - static_cast<int>(bits >> 23 & 255u);      // 150 or more: all of it lies below 2^-64 (zero among them)
  const unsigned __int128 window = right >= 128 ? 0 : right >= 0 ? kInv2Pi >> right : kInv2Pi << -right;
  const unsigned long long low = static_cast<uint32_t>(window), high = static_cast<unsigned long long>(window >> 32);
  const unsigned long long turns = m * high + (m * low >> 32);
  return bits >> 31 ? 0 - turns : turns;
}

template <typename T> struct Pack;
template <> struct Pack<__half> {
  static __device__ __forceinline__ float2 get(uint32_t w) { return __half22float2(*reinterpret_cast<__half2*>(&w)); }
  static __device__ __forceinline__ uint32_t put(float a, float b) {
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
};
template <> struct Pack<__nv_bfloat16> {
  static __device__ __forceinline__ float2 get(uint32_t w) {
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
  }
  static __device__ __forceinline__ uint32_t put(float a, float b) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
};
__device__ __forceinline__ float to_f(__half v) { return __half2float(v); }
__device__ __forceinline__ float to_f(__nv_bfloat16 v) { return __bfloat162float(v); }

// Two vectors of eight values, rotated: `half` pairs a[e] with b[e]; otherwise
// neighbours within each vector are pairs (a's first).
template <typename T>
__device__ __forceinline__ void rotate_half(uint4& a, uint4& b, const float2* cs) {
  uint32_t* pa = &a.x;
  uint32_t* pb = &b.x;
#pragma unroll
  for (int w = 0; w < 4; ++w) {
    const float2 x = Pack<T>::get(pa[w]), y = Pack<T>::get(pb[w]);
    const float2 c0 = cs[2 * w], c1 = cs[2 * w + 1];
    pa[w] = Pack<T>::put(x.x * c0.x - y.x * c0.y, x.y * c1.x - y.y * c1.y);
    pb[w] = Pack<T>::put(y.x * c0.x + x.x * c0.y, y.y * c1.x + x.y * c1.y);
  }
}
template <typename T>
__device__ __forceinline__ void rotate_adjacent(uint4& a, const float2* cs) {
  uint32_t* pa = &a.x;
#pragma unroll
  for (int w = 0; w < 4; ++w) {
    const float2 x = Pack<T>::get(pa[w]);
    const float2 c = cs[w];
    pa[w] = Pack<T>::put(x.x * c.x - x.y * c.y, x.y * c.x + x.x * c.y);
  }
}

// What one unit of work touches: up to two 16-byte vectors of one head of one token.
struct Unit {
  const char* src;
  char* dst;            // null: nothing to do (a token without a slot)
  int a, b;             // element offsets; b < 0: only a
  int pair;             // first pair of vector a (half) or of vectors a and b (adjacent); -1: copy
};

// kVec: pairs are whole 16-byte vectors (R % 8 == 0, or R % 4 == 0 with adjacent
// pairs) and a thread moves them by units. Otherwise 16 or 32 lanes take a head's row
// together, a vector each, and find the other halves of their pairs in shared memory.
template <typename T, bool kVec>
__global__ void __launch_bounds__(kRopeThreads) rope_kernel(const __grid_constant__ RopeKernelParams kp) {
  const RopeParams& p = kp.r;
  __shared__ float2 cs[kRopeMaxTokens * kRopeMaxPairs];
  __shared__ long long kbase[kRopeMaxTokens], vbase[kRopeMaxTokens];   // < 0: not stored
  const int t0 = static_cast<int>(blockIdx.x) * kp.tokens_per_cta;
  const int nt = min(kp.tokens_per_cta, p.tokens - t0);
  const int R = p.pairs;
  allow_dependents_launch();
  grid_dependency_wait();

  for (int i = threadIdx.x; i < nt * R; i += kRopeThreads) {
    const int t = i / R, pair = i - t * R;
    int axis = 0;
    while (axis + 1 < p.axes && pair >= p.section_end[axis]) ++axis;
    const unsigned long long frac = turns_of(p.inv_freq[pair]);
    const long long pos = p.positions[axis * p.pos_stride + t0 + t];
    const unsigned long long angle = frac * static_cast<unsigned long long>(pos);
    const float half_turns = static_cast<float>(static_cast<int32_t>(angle >> 32)) * 0x1p-31f;
    float s, c;
    sincospif(half_turns, &s, &c);
    cs[i] = make_float2(c, p.inverse ? -s : s);
  }
  if (p.kv_heads > 0 && threadIdx.x < nt) {
    const long long slot = p.slots[t0 + threadIdx.x];
    const bool stored = slot >= 0 && slot < static_cast<long long>(p.num_pages) * p.page_size;
    const long long page = stored ? slot / p.page_size : 0, at = stored ? slot % p.page_size : 0;
    kbase[threadIdx.x] = stored ? page * p.kc_ps + at * p.kc_ss : -1;
    vbase[threadIdx.x] = stored ? page * p.vc_ps + at * p.vc_ss : -1;
  }
  __syncthreads();

  const uint32_t per_token = kp.unit_div.d, rot = kp.rot_div.d, copy = kp.copy_div.d;
  const uint32_t total = static_cast<uint32_t>(nt) * per_token;
  const uint32_t rot_units = static_cast<uint32_t>(p.q_heads + p.kv_heads) * rot;

  auto unit = [&](uint32_t i) {
    Unit u;
    u.dst = nullptr;
    u.src = nullptr;
    u.a = 0;
    u.b = -1;
    u.pair = -1;
    const uint32_t t = kp.unit_div.div(static_cast<int>(i));
    uint32_t j = i - t * per_token;
    const long long tok = t0 + t;
    if (j < rot_units) {
      const uint32_t h = kp.rot_div.div(static_cast<int>(j));
      j -= h * rot;
      if (h < static_cast<uint32_t>(p.q_heads)) {
        u.src = reinterpret_cast<const char*>(static_cast<const T*>(p.q) + tok * p.q_ts + h * p.q_hs);
        u.dst = reinterpret_cast<char*>(static_cast<T*>(p.qo) + tok * p.qo_ts + h * p.qo_hs);
      } else {
        const long long kh = h - p.q_heads;
        if (kbase[t] < 0) return u;
        u.src = reinterpret_cast<const char*>(static_cast<const T*>(p.k) + tok * p.k_ts + kh * p.k_hs);
        u.dst = reinterpret_cast<char*>(static_cast<T*>(p.kc) + kbase[t] + kh * p.kc_hs);
      }
      const int jj = static_cast<int>(j);
      if (!kVec) {
        u.pair = static_cast<int>(t) * R;
      } else if (!p.interleaved) {
        const int nr = R / 8;
        if (jj < nr) {
          u.a = 8 * jj;
          u.b = R + 8 * jj;
          u.pair = static_cast<int>(t) * R + 8 * jj;
        } else {
          u.a = 2 * R + 16 * (jj - nr);
          u.b = u.a + 8 < p.dim ? u.a + 8 : -1;
        }
      } else {
        u.a = 16 * jj;
        u.b = u.a + 8 < p.dim ? u.a + 8 : -1;
        u.pair = u.a < 2 * R ? static_cast<int>(t) * R + 8 * jj : -1;
      }
    } else {
      j -= rot_units;
      const uint32_t h = kp.copy_div.div(static_cast<int>(j));
      j -= h * copy;
      if (vbase[t] < 0) return u;
      u.src = reinterpret_cast<const char*>(static_cast<const T*>(p.v) + tok * p.v_ts + h * p.v_hs);
      u.dst = reinterpret_cast<char*>(static_cast<T*>(p.vc) + vbase[t] + h * p.vc_hs);
      u.a = 16 * static_cast<int>(j);
      u.b = u.a + 8 < p.dim ? u.a + 8 : -1;
    }
    return u;
  };

  if constexpr (kVec) {
    for (uint32_t i = threadIdx.x; i < total; i += kRopeThreads) {
      const Unit u = unit(i);
      if (!u.dst) continue;
      uint4 a = *reinterpret_cast<const uint4*>(u.src + 2 * u.a), b;
      if (u.b >= 0) b = *reinterpret_cast<const uint4*>(u.src + 2 * u.b);
      if (u.pair >= 0) {
        if (!p.interleaved) {
          rotate_half<T>(a, b, cs + u.pair);
        } else {
          rotate_adjacent<T>(a, cs + u.pair);
          if (u.b >= 0 && u.b < 2 * R) rotate_adjacent<T>(b, cs + u.pair + 4);
        }
      }
      *reinterpret_cast<uint4*>(u.dst + 2 * u.a) = a;
      if (u.b >= 0) *reinterpret_cast<uint4*>(u.dst + 2 * u.b) = b;
    }
  } else {
    __shared__ __align__(16) T rows[kRopeThreads / 32][2 * kRopeMaxPairs];   // two rows of up to 128, or one
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int lanes = p.dim <= 128 ? 16 : 32, at_once = 32 / lanes;
    T* row = rows[warp] + (lane / lanes) * 128;
    const int e0 = lane % lanes * 8;
    for (uint32_t i0 = warp * at_once; i0 < total; i0 += kRopeThreads / 32 * at_once) {
      const uint32_t i = i0 + lane / lanes;     // (a unit is a whole row here)
      Unit u;
      u.dst = nullptr;
      if (i < total && e0 < p.dim) u = unit(i);
      uint4 v = make_uint4(0, 0, 0, 0);
      if (u.dst) {
        v = *reinterpret_cast<const uint4*>(u.src + 2 * e0);
        *reinterpret_cast<uint4*>(row + e0) = v;
      }
      __syncwarp();                              // the row has been read whole before any of it is written (in place)
      if (u.dst) {
        if (u.pair >= 0) {
          uint32_t* words = &v.x;
#pragma unroll
          for (int k = 0; k < 8; k += 2) {
            const float2 x = Pack<T>::get(words[k >> 1]);
            float y[2] = {x.x, x.y};
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const int e = e0 + k + i;
              if (e >= 2 * R) continue;
              const bool upper = p.interleaved ? i != 0 : e >= R;
              const int pair = p.interleaved ? e >> 1 : upper ? e - R : e;
              const float z = p.interleaved ? (i ? x.x : x.y) : to_f(row[upper ? e - R : e + R]);
              const float2 c = cs[u.pair + pair];
              y[i] = fmaf(y[i], c.x, upper ? z * c.y : -z * c.y);
            }
            words[k >> 1] = Pack<T>::put(y[0], y[1]);
          }
        }
        *reinterpret_cast<uint4*>(u.dst + 2 * e0) = v;
      }
      __syncwarp();
    }
  }
}

template <typename T>
cudaError_t launch(const RopeParams& r, int num_sms, cudaStream_t stream) {
  const RopeUnits u(r);
  const int per_token = static_cast<int>(u.per_token(r));
  // Tokens of a CTA: 4 or 2 where that still leaves every SM its eight CTAs (8192 tokens of
  // 48 heads: 37.3 us with 4 or 2, 42.2 with 1; 4099 of 32 heads: 15.3 with 2, 16.2 with 1, 16.8 with 4).
  int tokens = kRopeMaxTokens;
  while (tokens > 1 && r.tokens < 8 * num_sms * tokens) tokens >>= 1;
  const RopeKernelParams kp{r, FastDiv(per_token), FastDiv(u.rot), FastDiv(u.copy), tokens};
  const int grid = (r.tokens + tokens - 1) / tokens;
  return launch_dependent(u.vec ? rope_kernel<T, true> : rope_kernel<T, false>, grid, kRopeThreads, 0, stream, kp);
}

}  // namespace

cudaError_t launch_rope(FloatType t, const RopeParams& r, int num_sms, cudaStream_t stream) {
  return t == FloatType::BF16 ? launch<__nv_bfloat16>(r, num_sms, stream) : launch<__half>(r, num_sms, stream);
}

}  // namespace kaio
