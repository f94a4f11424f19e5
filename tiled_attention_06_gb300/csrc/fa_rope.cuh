// What the kernels that turn heads by their positions share: element types, angles as 64-bit
// fractions of a turn, the sequences of a CTA's tokens.
#pragma once

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
__device__ __forceinline__ void sequences_of(const int32_t* cu, int B, int T, uint32_t* status,
                                             int64_t t0, int nt, int* s_seq) {
  if (threadIdx.x < nt) s_seq[threadIdx.x] = kNobody;
  __syncthreads();
  for (int b = threadIdx.x; b < B; b += blockDim.x) {
    const SeqRows r = rows_of(cu, b, T);
    if (r.bad && blockIdx.x == 0) atomicOr(status, FA_DEV_BAD_PAGE);
    const int64_t end = static_cast<int64_t>(r.first) + r.n;
    for (int64_t t = max(t0, static_cast<int64_t>(r.first)); t < min(t0 + nt, end); ++t)
      atomicMin(s_seq + (t - t0), b);
  }
  __syncthreads();
}

}  // namespace
}  // namespace fa
