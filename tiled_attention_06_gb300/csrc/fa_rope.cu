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

#include <climits>
#include <cstdint>

#include "fa_varlen.h"
#include "fa_varlen_plan.cuh"

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

// Fraction of a turn per position, in units of 2^-64 turns: the double m 2^(e - 1075) times
// 2^64 / (2 pi), modulo 2^64, in integers (a chain of FP64 operations took 1.8 us of a decode
// step's 6). 2^66 / (2 pi) to 64 bits keeps the product good to 2^-62 of itself.
__device__ __forceinline__ uint64_t turns_q64(double radians) {
  constexpr uint64_t kTurns66 = 11743562013128004905ull;  // floor(2^66 / (2 pi))
  const uint64_t bits = static_cast<uint64_t>(__double_as_longlong(radians));
  const int e = static_cast<int>((bits >> 52) & 2047);
  if (e == 0 || e == 2047) return 0;  // zero (and what is too small to turn); not a frequency
  const uint64_t m = (bits & ((1ull << 52) - 1)) | (1ull << 52);
  const uint64_t lo = m * kTurns66, hi = __umul64hi(m, kTurns66);
  const int s = 1077 - e;  // right shift of hi:lo
  uint64_t t;
  if (s >= 128)
    t = 0;
  else if (s >= 64)
    t = hi >> (s - 64);
  else if (s > 0)
    t = (lo >> s) | (hi << (64 - s));
  else
    t = s > -64 ? lo << -s : 0;
  return bits >> 63 ? 0 - t : t;
}

// The sequences of tokens t0 .. t0 + nt - 1, found by the whole CTA: every sequence is asked, so
// that a bad start takes no token from another one. kNobody: no valid sequence owns the token.
constexpr int kNobody = INT_MAX;
__device__ __forceinline__ void sequences_of(const RopeParams& p, int64_t t0, int nt, int* s_seq) {
  if (threadIdx.x < nt) s_seq[threadIdx.x] = kNobody;
  __syncthreads();
  for (int b = threadIdx.x; b < p.B; b += kRopeThreads) {
    const SeqRows r = rows_of(p.cu, b, static_cast<int>(p.T));
    if (r.bad && blockIdx.x == 0) atomicOr(p.status, FA_DEV_BAD_PAGE);
    const int64_t end = static_cast<int64_t>(r.first) + r.n;
    for (int64_t t = max(t0, static_cast<int64_t>(r.first)); t < min(t0 + nt, end); ++t)
      atomicMin(s_seq + (t - t0), b);
  }
  __syncthreads();
}

// One CTA per `tok` tokens. A row (head) is cut into units of two chunks (of 16 bytes, or one
// element when VEC = 1): in the half layout chunks u and u + R/2, in the pair layout, in the
// unrotated rest and in copied rows neighbours. APPEND: rows 0 .. H-1 are q's, then Hkv of k's
// and Hkv of v's (copied). The units of the CTA's tokens are dealt to its threads in order; one
// unit in flight per thread and many threads did better than the reverse (16384 tokens x 40
// heads of 128 in bf16: 59.5 us, 5640 GB/s, against 71.6 with two in flight).
template <int DT, int VEC, bool HALF, bool APPEND>
__global__ void __launch_bounds__(kRopeThreads) rope_kernel(const RopeParams p, int tok) {
  using E = Elem<DT>;
  using T = typename E::T;
  using C = Chunk<T, VEC>;
  extern __shared__ float2 s_cs[];         // [tok][R/2] (cos, sin), amplitude included
  __shared__ int64_t s_dst[8];             // APPEND: first element of the token's slot, or below 0
  const int half = p.rot / 2;
  uint64_t* s_freq = reinterpret_cast<uint64_t*>(s_cs + static_cast<size_t>(tok) * half);
  const int64_t t0 = static_cast<int64_t>(blockIdx.x) * tok;
  const int nt = static_cast<int>(min(static_cast<int64_t>(tok), p.T - t0));
  for (int i = threadIdx.x; i < half; i += kRopeThreads) s_freq[i] = turns_q64(p.freqs[i]);
  __shared__ int64_t s_pos[8];  // a length near 2^31 and the chunk's tokens leave 32 bits
  if constexpr (APPEND) {
    __shared__ int s_seq[8];
    sequences_of(p, t0, nt, s_seq);
    if (threadIdx.x < nt) {
      const int64_t t = t0 + threadIdx.x;
      const int b = s_seq[threadIdx.x];
      int64_t dst = -2;
      int64_t pos = 0;
      if (b != kNobody) {
        const int64_t at = static_cast<int64_t>(p.ctx[b]) + (t - p.cu[b]);
        const int64_t lp = at / p.page_size;
        const bool in = p.ctx[b] >= 0 && lp < p.max_pages;
        const int phys = in ? p.block_table[static_cast<size_t>(b) * p.max_pages + lp] : -1;
        dst = -1;
        if (phys < 0 || phys >= p.num_pages)
          atomicOr(p.status, FA_DEV_BAD_PAGE);
        else
          dst = (static_cast<int64_t>(phys) * p.Hkv * p.page_size + (at - lp * p.page_size)) * p.d;
        pos = at;
      }
      s_pos[threadIdx.x] = pos;
      s_dst[threadIdx.x] = dst;  // -2: nobody's token, nothing is written; -1: no slot, q alone is
    }
  } else if (threadIdx.x < nt) {
    s_pos[threadIdx.x] = p.pos[t0 + threadIdx.x];
  }
  __syncthreads();
  for (int i = threadIdx.x; i < nt * half; i += kRopeThreads) {
    const int tk = i / half, f = i - tk * half;
    const int64_t at = p.inverse ? -s_pos[tk] : s_pos[tk];
    const uint64_t phase = static_cast<uint64_t>(at) * s_freq[f];
    float s, c;  // the phase as a signed fraction of a turn: half turns in [-1, 1]
    sincospif(static_cast<float>(static_cast<int64_t>(phase)) * 1.08420217248550443e-19f, &s, &c);
    s_cs[i] = make_float2(c * p.amplitude, s * p.amplitude);
  }
  __syncthreads();

  const int ru = half / VEC;                                       // rotated units of a row
  const int U = APPEND || p.copy_rest ? p.d / (2 * VEC) : ru;      // units of a row
  const int rows = APPEND ? p.H + 2 * p.Hkv : p.H;
  const int per_tok = rows * U, total = nt * per_tok;
  for (int j = threadIdx.x; j < total; j += kRopeThreads) {
    const int tk = j / per_tok, w = j - tk * per_tok, r = w / U, u = w - r * U;
    const int64_t t = t0 + tk;
    const T* src;
    T* dst;
    bool turn = u < ru;
    if (!APPEND || r < p.H) {
      if (APPEND && s_dst[tk] == -2) continue;
      src = static_cast<const T*>(p.x) + t * p.x_token + r * p.x_head;
      dst = static_cast<T*>(p.y) + t * p.y_token + r * p.y_head;
    } else {
      if (s_dst[tk] < 0) continue;
      const bool is_k = r < p.H + p.Hkv;
      const int h = r - p.H - (is_k ? 0 : p.Hkv);
      src = static_cast<const T*>(is_k ? p.k : p.v) + t * (is_k ? p.k_token : p.v_token) +
            static_cast<int64_t>(h) * p.d;
      dst = static_cast<T*>(is_k ? p.k_pages : p.v_pages) + s_dst[tk] +
              static_cast<int64_t>(h) * p.page_size * p.d;
      turn = turn && is_k;
    }
    // a copied row and the rest are cut alike: neighbours, the rest behind the rotated units
    const int oa = HALF && turn ? u * VEC : 2 * u * VEC, ob = HALF && turn ? half + oa : oa + VEC;
    C a = *reinterpret_cast<const C*>(src + oa), b = *reinterpret_cast<const C*>(src + ob);
    if (turn) {
      const float2* cs = s_cs + tk * half + u * VEC;
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        const float2 k = cs[e];
        // pair e of the unit: element e of both chunks, or neighbours 2e, 2e + 1 of the two
        constexpr bool kSplit = HALF || VEC == 1;
        T& xa = kSplit ? a.e[e] : (2 * e < VEC ? a.e[(2 * e) % VEC] : b.e[(2 * e) % VEC]);
        T& xb = kSplit ? b.e[e] : (2 * e < VEC ? a.e[(2 * e + 1) % VEC] : b.e[(2 * e + 1) % VEC]);
        const float fa = E::get(xa), fb = E::get(xb);
        xa = E::put(fa * k.x - fb * k.y);
        xb = E::put(fb * k.x + fa * k.y);
      }
    }
    *reinterpret_cast<C*>(dst + oa) = a;
    *reinterpret_cast<C*>(dst + ob) = b;
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
