// Rotary positions for packed tokens, and their fused form that also writes a paged cache.
//
// For a token at position p, pair i of the rotated part of a head (R elements, frequency
// w_i radians per position, amplitude A) is turned by t = p w_i:
//     y_a = A (x_a cos t - x_b sin t),   y_b = A (x_b cos t + x_a sin t),
// with (a, b) = (i, i + R/2) in the half layout and (2i, 2i + 1) in the pair layout;
// elements R .. d-1 pass through. The inverse call turns by -t: up to A it is the transpose,
// so it is the gradient of the forward call.
//
// Angles. p w_i reaches 10^6 radians in long contexts, where its FP32 product is off by 0.06
// rad. Each frequency is turned once per CTA into a 64-bit fixed-point fraction of a turn;
// p times it, modulo 2^64, is then the angle's fraction of a turn, exact for any 32-bit p up
// to the frequency's own rounding (2^-55 turns per position), in one integer multiplication.
//
// What bounds it: each element is read and written once for a handful of operations, so HBM
// does in bulk and latency in a decode step. A CTA takes a few tokens: it forms their sines
// and cosines once in shared memory for all heads, then streams the heads in 16-byte
// accesses. A token's sines cost R/2 sincospif, shared by its H + Hkv heads.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cstdint>

#include "fa_varlen.h"

namespace fa {
namespace {

constexpr int kRopeThreads = 256;

template <int DT>
struct Elem;
template <>
struct Elem<FA_F16> {
  using T = uint16_t;
  static __device__ __forceinline__ float get(T v) { return __half2float(__ushort_as_half(v)); }
  static __device__ __forceinline__ T put(float f) { return __half_as_ushort(__float2half_rn(f)); }
};
template <>
struct Elem<FA_BF16> {
  using T = uint16_t;
  static __device__ __forceinline__ float get(T v) {
    return __uint_as_float(static_cast<uint32_t>(v) << 16);
  }
  static __device__ __forceinline__ T put(float f) {
    return __bfloat16_as_ushort(__float2bfloat16_rn(f));
  }
};
template <>
struct Elem<FA_F32> {
  using T = float;
  static __device__ __forceinline__ float get(T v) { return v; }
  static __device__ __forceinline__ T put(float f) { return f; }
};

// VEC consecutive elements as one access (VEC elements are 16 bytes, or VEC = 1).
template <typename T, int VEC>
struct alignas(sizeof(T) * VEC) Chunk {
  T e[VEC];
};

// Fraction of a turn per position, in units of 2^-64 turns. Once per frequency and CTA.
__device__ __forceinline__ uint64_t turns_q64(double radians) {
  const double t = radians * 0.15915494309189533577;  // 1 / (2 pi)
  const double f = t - floor(t);
  return f >= 1.0 ? 0ull : __double2ull_rz(f * 18446744073709551616.0);
}

// The sequence of token t: the number of sequences that end at or before it (cu holds B + 1
// non-decreasing starts), counted by the whole CTA.
__device__ __forceinline__ int sequence_of(const int32_t* cu, int B, int64_t t) {
  int n = 0;
  for (int i0 = 0; i0 < B; i0 += kRopeThreads) {
    const int i = i0 + threadIdx.x;
    n += __syncthreads_count(i < B && cu[i + 1] <= t);
  }
  return n;
}

// One CTA per `tok` tokens. A row (head) is cut into units. VEC > 1: in the half layout a unit
// is the two 16-byte chunks u and u + R/2, or one chunk of the unrotated rest; in the pair
// layout one chunk. VEC = 1: one pair, or one element of the rest. APPEND: rows 0 .. H-1 are
// q's, then Hkv of k's; v's rows are copied.
template <int DT, int VEC, bool HALF, bool APPEND>
__global__ void __launch_bounds__(kRopeThreads, 3) rope_kernel(const RopeParams p, int tok) {
  using E = Elem<DT>;
  using T = typename E::T;
  using C = Chunk<T, VEC>;
  constexpr bool kTwo = HALF || VEC == 1;  // a rotated unit holds two chunks
  constexpr int kAngles = kTwo ? VEC : VEC / 2;  // angles of a rotated unit
  extern __shared__ float2 s_cs[];         // [tok][R/2] (cos, sin), amplitude included
  __shared__ int64_t s_dst[8];             // APPEND: first element of the token's slot, or -1
  const int half = p.rot / 2;
  uint64_t* s_freq = reinterpret_cast<uint64_t*>(s_cs + static_cast<size_t>(tok) * half);
  const int64_t t0 = static_cast<int64_t>(blockIdx.x) * tok;
  const int nt = static_cast<int>(min(static_cast<int64_t>(tok), p.T - t0));
  for (int i = threadIdx.x; i < half; i += kRopeThreads) s_freq[i] = turns_q64(p.freqs[i]);
  __shared__ int s_pos[8];
  if constexpr (APPEND) {
    const int b0 = sequence_of(p.cu, p.B, t0);
    if (threadIdx.x < nt) {  // a later token of the CTA may belong to a later sequence
      const int64_t t = t0 + threadIdx.x;
      int b = b0;
      while (b < p.B && p.cu[b + 1] <= t) ++b;
      int64_t dst = -1;
      int pos = 0;
      if (b < p.B && p.cu[b] <= t) {
        const int64_t at = static_cast<int64_t>(p.ctx[b]) + (t - p.cu[b]);
        const int64_t lp = at / p.page_size;
        const bool in = p.ctx[b] >= 0 && lp < p.max_pages;
        const int phys = in ? p.block_table[static_cast<size_t>(b) * p.max_pages + lp] : -1;
        if (phys < 0 || phys >= p.num_pages)
          atomicOr(p.status, FA_DEV_BAD_PAGE);
        else
          dst = (static_cast<int64_t>(phys) * p.Hkv * p.page_size + (at - lp * p.page_size)) * p.d;
        pos = static_cast<int>(at);
      }
      s_pos[threadIdx.x] = pos;
      // -2: behind the last sequence, nothing is written; -1: no slot, q alone is
      s_dst[threadIdx.x] = (b < p.B && p.cu[b] <= t) ? dst : -2;
    }
  } else if (threadIdx.x < nt) {
    s_pos[threadIdx.x] = p.pos[t0 + threadIdx.x];
  }
  __syncthreads();
  for (int i = threadIdx.x; i < nt * half; i += kRopeThreads) {
    const int tk = i / half, f = i - tk * half;
    const int64_t at = p.inverse ? -static_cast<int64_t>(s_pos[tk]) : s_pos[tk];
    const uint64_t phase = static_cast<uint64_t>(at) * s_freq[f];
    float s, c;  // the phase as a signed fraction of a turn: half turns in [-1, 1]
    sincospif(static_cast<float>(static_cast<int64_t>(phase)) * 1.08420217248550443e-19f, &s, &c);
    s_cs[i] = make_float2(c * p.amplitude, s * p.amplitude);
  }
  __syncthreads();

  // A thread keeps one unit, its angles in registers, and takes every `step`-th row of one token
  // (or of several, when a row has so many units that the CTA covers fewer tokens at once).
  const int ru = half / kAngles;                           // rotated units of a row
  const int rest = (p.copy_rest ? p.d - p.rot : 0) / VEC;  // units of the unrotated rest
  const int vu = kTwo && VEC > 1 ? p.d / (2 * VEC) : p.d / VEC;  // units of a copied row
  const int U = APPEND ? max(ru + rest, vu) : ru + rest;
  const int lu = min(U, kRopeThreads), groups = kRopeThreads / lu;
  const int g = threadIdx.x / lu, gt = min(tok, groups), step = groups / gt;
  if (g >= gt * step) return;
  const int turned = APPEND ? p.H + p.Hkv : p.H;
  for (int tk = g / step; tk < nt; tk += gt) {  // lanes next to each other: rows of one token
    const int64_t t = t0 + tk;
    const int64_t slot = APPEND ? s_dst[tk] : 0;
    if (APPEND && slot == -2) continue;
    for (int u = threadIdx.x - g * lu; u < U; u += lu) {
      // first elements of the unit's chunks
      const bool rot = u < ru;
      int oa, ob = 0;
      if (!rot) {
        oa = p.rot + (u - ru) * VEC;
      } else if (VEC == 1) {
        oa = HALF ? u : 2 * u;
        ob = HALF ? half + u : 2 * u + 1;
      } else {
        oa = u * VEC;
        ob = half + u * VEC;
      }
      float2 cs[kAngles];
      if (rot) {
#pragma unroll
        for (int e = 0; e < kAngles; ++e) cs[e] = s_cs[tk * half + u * kAngles + e];
      }
      auto src_of = [&](int r) -> const T* {
        if (APPEND && r >= p.H)
          return static_cast<const T*>(p.k) + t * p.k_token + static_cast<int64_t>(r - p.H) * p.d;
        return static_cast<const T*>(p.x) + t * p.x_token + r * p.x_head;
      };
      auto dst_of = [&](int r) -> T* {
        if (APPEND && r >= p.H)
          return static_cast<T*>(p.k_pages) + slot +
                 static_cast<int64_t>(r - p.H) * p.page_size * p.d;
        return static_cast<T*>(p.y) + t * p.y_token + r * p.y_head;
      };
      const int rows = APPEND && slot < 0 ? p.H : turned;  // no slot: q alone
      constexpr int N = 2;                                 // rows in flight
      for (int r0 = g % step; r0 < rows && u < ru + rest; r0 += N * step) {
        C a[N], b[N];
#pragma unroll
        for (int i = 0; i < N; ++i) {
          const int r = r0 + i * step;
          if (r < rows) {
            a[i] = *reinterpret_cast<const C*>(src_of(r) + oa);
            if (kTwo && rot) b[i] = *reinterpret_cast<const C*>(src_of(r) + ob);
          }
        }
#pragma unroll
        for (int i = 0; i < N; ++i) {
          const int r = r0 + i * step;
          if (r >= rows) break;
          if (rot) {
            if constexpr (kTwo) {
#pragma unroll
              for (int e = 0; e < VEC; ++e) {
                const float xa = E::get(a[i].e[e]), xb = E::get(b[i].e[e]);
                a[i].e[e] = E::put(xa * cs[e].x - xb * cs[e].y);
                b[i].e[e] = E::put(xb * cs[e].x + xa * cs[e].y);
              }
              *reinterpret_cast<C*>(dst_of(r) + ob) = b[i];
            } else {
#pragma unroll
              for (int e = 0; e < kAngles; ++e) {
                const float xa = E::get(a[i].e[2 * e]), xb = E::get(a[i].e[2 * e + 1]);
                a[i].e[2 * e] = E::put(xa * cs[e].x - xb * cs[e].y);
                a[i].e[2 * e + 1] = E::put(xb * cs[e].x + xa * cs[e].y);
              }
            }
          }
          *reinterpret_cast<C*>(dst_of(r) + oa) = a[i];
        }
      }
      if constexpr (APPEND) {
        for (int r = g % step; r < p.Hkv && u < vu && slot >= 0; r += step) {
          const T* src = static_cast<const T*>(p.v) + t * p.v_token + static_cast<int64_t>(r) * p.d;
          T* dst = static_cast<T*>(p.v_pages) + slot + static_cast<int64_t>(r) * p.page_size * p.d;
          const C a = *reinterpret_cast<const C*>(src + u * VEC);
          if constexpr (kTwo && VEC > 1) {
            const C b = *reinterpret_cast<const C*>(src + p.d / 2 + u * VEC);
            *reinterpret_cast<C*>(dst + p.d / 2 + u * VEC) = b;
          }
          *reinterpret_cast<C*>(dst + u * VEC) = a;
        }
      }
    }
  }
}

template <int DT, bool APPEND>
cudaError_t launch_rope_t(const RopeParams& p, bool half_style, bool vec, int sms,
                          cudaStream_t stream) {
  // Tokens per CTA: one while that leaves SMs without work (a decode step), four for a prompt.
  const int tok = p.T >= 16LL * sms ? 4 : 1;
  const size_t smem = static_cast<size_t>(p.rot / 2) * (tok * sizeof(float2) + sizeof(uint64_t));
  const int64_t grid = (p.T + tok - 1) / tok;
  if (grid > 0x7fffffff) return cudaErrorInvalidConfiguration;
  constexpr int V = DT == FA_F32 ? 4 : 8;
  auto* k = vec ? (half_style ? rope_kernel<DT, V, true, APPEND> : rope_kernel<DT, V, false, APPEND>)
                : (half_style ? rope_kernel<DT, 1, true, APPEND> : rope_kernel<DT, 1, false, APPEND>);
  k<<<static_cast<unsigned>(grid), kRopeThreads, smem, stream>>>(p, tok);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_rope(const RopeParams& p, int dtype, bool half_style, bool vec, int sms,
                        cudaStream_t stream) {
  if (dtype == FA_F32) return launch_rope_t<FA_F32, false>(p, half_style, vec, sms, stream);
  if (dtype == FA_BF16) return launch_rope_t<FA_BF16, false>(p, half_style, vec, sms, stream);
  return launch_rope_t<FA_F16, false>(p, half_style, vec, sms, stream);
}

cudaError_t launch_rope_append(const RopeParams& p, int dtype, bool half_style, bool vec, int sms,
                               cudaStream_t stream) {
  if (dtype == FA_BF16) return launch_rope_t<FA_BF16, true>(p, half_style, vec, sms, stream);
  return launch_rope_t<FA_F16, true>(p, half_style, vec, sms, stream);
}

}  // namespace fa
