// Norms of query and key heads with rotary positions of one or several axes in the same pass, the
// gradient, and the form that writes a paged cache in 16 or 8 bits.
//
// For a head x of d elements, weight w and a token with positions p_0 .. p_{A-1} (A axes, say
// time, height and width), with pair i of the rotated part turned by t_i = p_{axis(i)} w_i:
//     n = x r w,  r = 1 / sqrt(mean(x^2) + eps),      y = R(t) n   (fa_rope.cu's rotation),
// and for an upstream gradient dy, with g = R(t)^T dy:
//     dw = sum over tokens and heads of g x r,        dx = r w g - x r^3 mean(w g x).
// Everything between the load and the one rounding at the store is FP32.
//
// An 8-bit cache holds a row (one token and head) as d floats of 4 exponent and 3 mantissa bits
// times one power of two 2^e, e the smallest integer with max|y| <= 448 2^e, kept as the byte
// e + 127. A power of two costs such floats nothing but the lowest of their range, and values
// times it are exact in 16 bits, so what reads the cache rounds nothing. A row with an infinity or
// a NaN gets byte 255 and is NaN when read.
//
// What bounds it: each element is read once and written once (the gradient reads x and dy), so
// HBM does in bulk and latency in a decode step; on the way there, instructions. A row is spread over
// LN neighbouring lanes, 16 elements to a lane, whose sums meet in log2(LN) shuffles. A group of lanes
// keeps to one head and walks over the tokens of its CTA, so that its pointers advance by a constant, its
// weight stays in registers and the weight's gradient adds up there; arithmetic is in packed FP32, and
// rows come three rounds ahead by cp.async. With rows dealt to groups in order, whatever their token and
// head, addresses and weights cost a row more instructions than its arithmetic and 16384 tokens x 40
// heads of 128 in bf16 took 68 us and their gradient 117; so they take 62.8 (5340 GB/s, 80 % of the
// measured copy rate) and 95.8 (5250 GB/s). FP32, 8192 tokens x 40 heads of 64: 29.9 and 59.7 (floors 25.1
// and 37.7). Halves of the rotated part that are no multiple of 16 bytes move in
// chunks of 8 or 4 (8192 tokens, 72 or 68 of 128 elements rotated: 57 us element by element, 33 and 39).
#include <algorithm>
#include <climits>
#include <cstdint>
#include <type_traits>

#include "fa_ptx.cuh"
#include "fa_rope.cuh"

namespace fa {
namespace {

constexpr int kTokMax = 32;  // tokens of a batch at most
constexpr int kMostThreads = 320;
constexpr uint32_t kAll = 0xffffffffu;

// The exponent byte of a row from the bits of its largest magnitude: bits of an infinity or NaN
// give 255. 448 = 1.75 * 2^8, and a float m 2^(E - 127) has fraction bits 0x600000 at m = 1.75.
__device__ __forceinline__ int power_byte(uint32_t bits) {
  if (bits >= 0x7f800000u) return 255;
  const int e = static_cast<int>(bits >> 23) - 8 + ((bits & 0x7fffffu) > 0x600000u ? 1 : 0);
  return e < 0 ? 0 : e;
}
// 2^(127 - b): what brings the row within range (b <= 254 - 7, as no float has a higher exponent).
__device__ __forceinline__ float up_of(int b) {
  return __uint_as_float(static_cast<uint32_t>(254 - b) << 23);
}
// 2^(b - 127), NaN for 255
__device__ __forceinline__ float power_of(int b) {
  return __uint_as_float(b == 255 ? 0x7fffffffu : b == 0 ? 0x400000u
                                                          : static_cast<uint32_t>(b) << 23);
}
// Two floats to two 8-bit ones, `lo` in the low byte; to nearest, ties to even.
__device__ __forceinline__ uint32_t cvt_e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}
// Two 8-bit floats to two floats.
__device__ __forceinline__ float2 e4m3x2_to_f32(uint32_t x) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(static_cast<uint16_t>(x)));
  return __half22float2(*reinterpret_cast<__half2*>(&h));
}

// Where a lane's elements lie in a row: unit u holds VEC elements at oa and VEC at ob. In the half
// layout the rotated units are chunks u and u + R/2, every other unit neighbours.
template <int VEC, bool HALF>
__device__ __forceinline__ void unit_at(int u, int ru, int half, int& oa, int& ob) {
  const bool split = HALF && u < ru;
  oa = split ? u * VEC : 2 * u * VEC;
  ob = split ? half + oa : oa + VEC;
}

// A unit's elements go by VEC pairs (A_e, B_e), which the rotation turns: elements e of both chunks,
// or neighbours 2e and 2e + 1 of the two where pairs are neighbours (VEC > 1). Arithmetic takes two
// pairs at a time, (A_e, A_{e+1}) and (B_e, B_{e+1}), in packed FP32: of one unit, or where units are
// pairs (VEC = 1) of two of the lane's units.
//
// A CTA's shared memory: rows on their way, sines and cosines of a batch of its tokens, the frequencies
// and the pairs' axes. For VEC > 1 the cosines and sines of two pairs are 16 bytes, neighbouring units
// next to each other, so that neighbouring lanes read neighbouring 16 bytes.
struct Shared {
  float2* cs;
  uint64_t* freq;
  uint8_t* axis;
  __device__ __forceinline__ Shared(float4* base, int pairs, int half) {
    cs = reinterpret_cast<float2*>(base);
    freq = reinterpret_cast<uint64_t*>(cs + pairs);
    axis = reinterpret_cast<uint8_t*>(freq + half);
  }
};
int shared_bytes(int pairs, int half) { return pairs * 8 + half * 9; }
// Rows on their way: every thread copies its own chunks of the rows to come to shared memory
// (cp.async) and reads them back itself, so nothing waits for anyone else. In registers a row ahead is
// what there is room for, 32 KB per SM on their way.
constexpr int kStages = 4;
// Rounds of x and dy; FP32's are twice as large, and with three of them one CTA is all that fits an SM
// (8192 tokens x 40 heads of 64: 70 us, 60 with two).
constexpr int grad_stages(int chunks) { return chunks == 1 ? 3 : 2; }
template <int N>
__device__ __forceinline__ void copy_async(uint32_t dst, const void* src) {
  if constexpr (N == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(dst), "l"(src), "n"(N) : "memory");
}
__device__ __forceinline__ void copy_commit() {
  asm volatile("cp.async.commit_group;" ::: "memory");
}
template <int N>
__device__ __forceinline__ void copy_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Where the cosine of pair e of unit u lies (its sine is two behind it for VEC > 1, one for VEC = 1),
// `units` rotated units in all: [e / 2][u][c_e c_{e+1} s_e s_{e+1}], or [u][c s].
template <int VEC>
__device__ __forceinline__ int pair_at(int u, int e, int units) {
  return VEC == 1 ? 2 * u : ((e / 2) * units + u) * 4 + e % 2;
}

// What a CTA reads before its first row: the frequencies and axes, and the first batch's positions, a
// thread's first of each in registers, so that these loads and the weights' wait for memory once.
struct Ahead {
  double freq = 0;
  int axis = 0, pos = 0;
  __device__ __forceinline__ void load(const NormRopeParams& p, int64_t t0, int nt) {
    const int i = threadIdx.x;
    if (i < p.rot / 2) {
      freq = p.freqs[i];
      if (p.pair_axis) axis = p.pair_axis[i];
    }
    if (p.pos && i < nt * p.axes) pos = p.pos[(i / nt) * p.T + t0 + i % nt];
  }
};
// Frequencies and axes, and the pairs behind the last rotated one that share its unit (neighbours):
// the part that does not depend on the tokens.
template <int VEC>
__device__ __forceinline__ void fill_fixed(const NormRopeParams& p, const Shared& sh,
                                           const Ahead& first, int tok, int slots) {
  const int rest = slots - p.rot / 2;
  for (int i = threadIdx.x; i < tok * rest; i += blockDim.x) {
    const int tk = i / rest, f = p.rot / 2 + i - tk * rest;
    float* const to =
        reinterpret_cast<float*>(sh.cs + tk * slots) + pair_at<VEC>(f / VEC, f % VEC, slots / VEC);
    to[0] = 1.f;
    to[VEC == 1 ? 1 : 2] = 0.f;
  }
  for (int i = threadIdx.x; i < p.rot / 2; i += blockDim.x) {
    const bool mine = i == static_cast<int>(threadIdx.x);
    sh.freq[i] = turns_q64(mine ? first.freq : p.freqs[i]);
    int a = mine ? first.axis : p.pair_axis ? p.pair_axis[i] : 0;
    if (a < 0 || a >= p.axes) {
      if (blockIdx.x == 0) atomicOr(p.status, FA_DEV_BAD_PAGE);
      a = 0;
    }
    sh.axis[i] = static_cast<uint8_t>(a);
  }
}
// The positions of the nt tokens from t0 on.
__device__ __forceinline__ void fill_positions(const NormRopeParams& p, int64_t (*s_pos)[kTokMax],
                                               int64_t t0, int nt, bool first, const Ahead& ahead) {
  for (int i = threadIdx.x; i < nt * p.axes; i += blockDim.x)
    s_pos[i / nt][i % nt] = first && i == static_cast<int>(threadIdx.x)
                                ? ahead.pos
                                : p.pos[(i / nt) * p.T + t0 + i % nt];
}
// Sines and cosines of nt tokens; pos(axis, token) in 64 bits.
template <int VEC, typename Pos>
__device__ __forceinline__ void fill_angles(const NormRopeParams& p, int nt, const Shared& sh, int slots,
                                            bool inverse, Pos pos) {
  const int half = p.rot / 2, ru = slots / VEC;
  const int dt = blockDim.x / half, df = blockDim.x % half;
  int tk = threadIdx.x / half, f = threadIdx.x % half;
  while (tk < nt) {
    const int64_t at = pos(sh.axis[f], tk);
    const uint64_t phase = static_cast<uint64_t>(inverse ? -at : at) * sh.freq[f];
    float s, c;  // the phase as a signed fraction of a turn: half turns in [-1, 1]
    sincospif(static_cast<float>(static_cast<int64_t>(phase)) * 1.08420217248550443e-19f, &s, &c);
    float* const to = reinterpret_cast<float*>(sh.cs + tk * slots) + pair_at<VEC>(f / VEC, f % VEC, ru);
    to[0] = c * p.amplitude;
    to[VEC == 1 ? 1 : 2] = s * p.amplitude;
    tk += dt;
    f += df;
    if (f >= half) {
      f -= half;
      ++tk;
    }
  }
}

__device__ __forceinline__ float f2_sum(uint64_t a) {
  float x, y;
  f2_split(a, x, y);
  return x + y;
}

template <typename C>
__device__ __forceinline__ C load_chunk(uint32_t at) {
  C c;
  if constexpr (sizeof(C) == 16) {
    uint32_t r[4];
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(at)
                 : "memory");
    __builtin_memcpy(&c, r, 16);
  } else if constexpr (sizeof(C) == 8) {
    uint32_t r[2];
    asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(r[0]), "=r"(r[1]) : "r"(at) : "memory");
    __builtin_memcpy(&c, r, 8);
  } else if constexpr (sizeof(C) == 4) {
    uint32_t r;
    asm volatile("ld.shared.b32 %0, [%1];" : "=r"(r) : "r"(at) : "memory");
    __builtin_memcpy(&c, &r, 4);
  }
  return c;
}

// A lane's part of a row: KU units of VEC + VEC elements; N pairs, worked on two at a time.
template <int DT, int VEC, int KU, bool HALF>
struct Part {
  using T = typename Elem<DT>::T;
  using C = Chunk<T, VEC>;
  static constexpr int N = KU * VEC, N2 = N / 2;
  C a[KU], b[KU];
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int k = 0; k < KU; ++k)
#pragma unroll
      for (int e = 0; e < VEC; ++e) a[k].e[e] = b[k].e[e] = T(0);
  }
  __device__ __forceinline__ void load(const T* src, const int* oa, const int* ob, int have) {
#pragma unroll
    for (int k = 0; k < KU; ++k)
      if (k < have) {
        a[k] = *reinterpret_cast<const C*>(src + oa[k]);
        b[k] = *reinterpret_cast<const C*>(src + ob[k]);
      }
  }
  // the same by way of shared memory: chunk c of the thread at c * step
  static __device__ __forceinline__ void fetch(uint32_t at, uint32_t step, const T* src,
                                               const int* oa, const int* ob, int have) {
#pragma unroll
    for (int k = 0; k < KU; ++k)
      if (k < have) {
        copy_async<sizeof(C)>(at + (2 * k) * step, src + oa[k]);
        copy_async<sizeof(C)>(at + (2 * k + 1) * step, src + ob[k]);
      }
  }
  // (a chunk that the row does not have is whatever lies there; its elements are zeroed)
  __device__ __forceinline__ void take(uint32_t at, uint32_t step, int have) {
#pragma unroll
    for (int k = 0; k < KU; ++k) {
      a[k] = load_chunk<C>(at + (2 * k) * step);
      b[k] = load_chunk<C>(at + (2 * k + 1) * step);
      if (k >= have) {
#pragma unroll
        for (int e = 0; e < VEC; ++e) a[k].e[e] = b[k].e[e] = T(0);
      }
    }
  }
  __device__ __forceinline__ T& first(int i) {
    const int k = i / VEC, e = i % VEC;
    if (HALF || VEC == 1) return a[k].e[e];
    return 2 * e < VEC ? a[k].e[(2 * e) % VEC] : b[k].e[(2 * e) % VEC];
  }
  __device__ __forceinline__ T& second(int i) {
    const int k = i / VEC, e = i % VEC;
    if (HALF || VEC == 1) return b[k].e[e];
    return 2 * e < VEC ? a[k].e[(2 * e + 1) % VEC] : b[k].e[(2 * e + 1) % VEC];
  }
  __device__ __forceinline__ void widen(uint64_t* A, uint64_t* B) {
#pragma unroll
    for (int i = 0; i < N2; ++i) {
      A[i] = f2(Elem<DT>::get(first(2 * i)), Elem<DT>::get(first(2 * i + 1)));
      B[i] = f2(Elem<DT>::get(second(2 * i)), Elem<DT>::get(second(2 * i + 1)));
    }
  }
  static __device__ __forceinline__ void store(T* dst, const int* oa, const int* ob, int have,
                                               const uint64_t* A, const uint64_t* B) {
    Part x;
#pragma unroll
    for (int i = 0; i < N2; ++i) {
      float u, v;
      f2_split(A[i], u, v);
      x.first(2 * i) = Elem<DT>::put(u);
      x.first(2 * i + 1) = Elem<DT>::put(v);
      f2_split(B[i], u, v);
      x.second(2 * i) = Elem<DT>::put(u);
      x.second(2 * i + 1) = Elem<DT>::put(v);
    }
#pragma unroll
    for (int k = 0; k < KU; ++k)
      if (k < have) {
        *reinterpret_cast<C*>(dst + oa[k]) = x.a[k];
        *reinterpret_cast<C*>(dst + ob[k]) = x.b[k];
      }
  }
};

// Cosines and sines of the lane's packed pair i, (c_e, c_{e+1}) and (s_e, s_{e+1}); its units are u0,
// u0 + ln, .... A unit behind the rotated part reads the last one's.
template <int VEC>
__device__ __forceinline__ void angles_of(const float* at, int i, int u0, int ln, int units,
                                          uint64_t& c, uint64_t& s) {
  if constexpr (VEC == 1) {
    const float2 x = *reinterpret_cast<const float2*>(at + 2 * min(u0 + 2 * i * ln, units - 1));
    const float2 y = *reinterpret_cast<const float2*>(at + 2 * min(u0 + (2 * i + 1) * ln, units - 1));
    c = f2(x.x, y.x);
    s = f2(x.y, y.y);
  } else {
    const int u = min(u0 + (2 * i / VEC) * ln, units - 1);
    const ulonglong2 x =
        *reinterpret_cast<const ulonglong2*>(at + pair_at<VEC>(u, 2 * i % VEC, units));
    c = x.x;
    s = x.y;
  }
}
// The rotation of a lane's pairs, (A, B) to (A c - B s, B c + A s), with nB = -B; those behind the
// rotated part stay.
template <int VEC, int N2, bool RAGGED>
__device__ __forceinline__ void turn(uint64_t* A, uint64_t* B, const uint64_t* nB, const float2* cs,
                                     int u0, int ln, int ru, int half) {
#pragma unroll
  for (int i = 0; i < N2; ++i) {
    uint64_t c, s;
    angles_of<VEC>(reinterpret_cast<const float*>(cs), i, u0, ln, ru, c, s);
    if (VEC > 1 && u0 + (2 * i / VEC) * ln >= ru) continue;
    const uint64_t a = A[i], b = B[i];
    A[i] = f2_fma(a, c, f2_mul(nB[i], s));
    B[i] = f2_fma(b, c, f2_mul(a, s));
    // pairs behind the last rotated one stay as they are, infinities too: the second of two units, or
    // neighbours that share its unit
    if (VEC == 1 || RAGGED) {
      const int in = VEC == 1 ? (u0 + 2 * i * ln < ru) + (u0 + (2 * i + 1) * ln < ru)
                              : half - (u0 + (2 * i / VEC) * ln) * VEC - 2 * i % VEC;
      const uint64_t keep = in < 1 ? ~0ull : in < 2 ? ~0ull << 32 : 0ull;
      A[i] = (A[i] & ~keep) | (a & keep);
      B[i] = (B[i] & ~keep) | (b & keep);
    }
  }
}
// The weights of a lane's elements, as its pairs lie; 0 where the row has no element. All loads of a
// kind of weight stand before their uses (one by one, each behind the question of which kind it is, they
// took 3.5 us of every CTA).
template <int DT, int VEC, int KU, bool HALF>
__device__ __forceinline__ void weights_of(const NormRopeParams& p, const void* w, const int* oa,
                                           const int* ob, int have, uint64_t* A, uint64_t* B) {
  constexpr int N = KU * VEC;
  int at[2][N];
#pragma unroll
  for (int n = 0; n < N; ++n) {
    const int k = n / VEC, e = n % VEC;
#pragma unroll
    for (int h = 0; h < 2; ++h)
      at[h][n] = k >= have                 ? -1
                 : HALF || VEC == 1 ? (h ? ob[k] : oa[k]) + e
                                    : oa[k] + 2 * e + h;
  }
  float v[2][N];
  if (!w) {
#pragma unroll
    for (int n = 0; n < 2 * N; ++n) v[n / N][n % N] = at[n / N][n % N] < 0 ? 0.f : 1.f;
  } else if (DT == FA_F32 || p.w_f32) {
#pragma unroll
    for (int n = 0; n < 2 * N; ++n) {
      const int i = at[n / N][n % N];
      const float x = static_cast<const float*>(w)[max(i, 0)];
      v[n / N][n % N] = i < 0 ? 0.f : x;
    }
  } else {
    uint16_t x[2][N];
#pragma unroll
    for (int n = 0; n < 2 * N; ++n)
      x[n / N][n % N] = static_cast<const uint16_t*>(w)[max(at[n / N][n % N], 0)];
#pragma unroll
    for (int n = 0; n < 2 * N; ++n) {
      const float f = DT == FA_BF16 ? Elem<FA_BF16>::get(x[n / N][n % N])
                                    : Elem<FA_F16>::get(x[n / N][n % N]);
      v[n / N][n % N] = at[n / N][n % N] < 0 ? 0.f : f;
    }
  }
#pragma unroll
  for (int i = 0; i < N / 2; ++i) {
    A[i] = f2(v[0][2 * i], v[0][2 * i + 1]);
    B[i] = f2(v[1][2 * i], v[1][2 * i + 1]);
  }
}
__device__ __forceinline__ float sum_lanes(float x, int ln) {
  for (int o = ln / 2; o > 0; o /= 2) x += __shfl_xor_sync(kAll, x, o);
  return x;
}

// How the rows are dealt. A CTA has a run of tokens and `heads` heads from blockIdx.y * heads on; group
// g of its lanes has head g % heads of tokens g / heads, g / heads + per_round, ... of the run. Angles are
// made for `tok` tokens (a multiple of per_round) at a time.
struct Deal {
  int ln, heads, per_round, tok;
};
struct Mine {
  int tr, r;           // first token of the run, head
  bool on;             // this group has a head
  int64_t begin, end;  // the CTA's tokens
  __device__ __forceinline__ Mine(const NormRopeParams& p, const Deal& d, int rows) {
    const int g = threadIdx.x / d.ln;
    tr = g / d.heads;
    r = blockIdx.y * d.heads + g - tr * d.heads;
    on = tr < d.per_round && r < rows;
    begin = p.T * blockIdx.x / gridDim.x;
    end = p.T * (blockIdx.x + 1) / gridDim.x;
  }
};

// Three of 64 registers a thread (8 to 12 bytes of them spilled) where those do; with the cache's addresses and bytes they spill (chunks
// of 8 sequences of up to 512 tokens, 8 bits: 14.9 us, 13.6 with two).
constexpr int ctas_per_sm(int dt, int vec, int mode) {
  return dt != FA_F32 && vec == 8 && mode == 0 ? 3 : 2;
}

// Rows r of a token: H of q, Hkv of k and, when appending, Hkv of v. MODE 0: y to q_out and k_out;
// 1 and 2: q to q_out, k and v to the cache's slot of the token, in 16 and in 8 bits.
template <int DT, int VEC, int KU, bool HALF, bool RAGGED, int MODE>
__global__ void __launch_bounds__(kMostThreads, ctas_per_sm(DT, VEC, MODE))
    norm_rope_kernel(const __grid_constant__ NormRopeParams p, const Deal deal) {
  using T = typename Elem<DT>::T;
  using X = Part<DT, VEC, KU, HALF>;
  constexpr int N2 = X::N2;
  extern __shared__ float4 s_dyn[];
  __shared__ int64_t s_dst[kTokMax], s_pos[FA_MAX_AXES][kTokMax];
  __shared__ int s_seq[kTokMax];
  const int half = p.rot / 2, ru = (half + VEC - 1) / VEC, slots = ru * VEC;
  const int U = p.d / (2 * VEC), ln = deal.ln;
  // chunk c of round i of the thread at ((i % kStages) * 2 KU + c) * step
  constexpr int CB = sizeof(typename X::C);  // bytes of a chunk
  const uint32_t step = blockDim.x * CB, stage = 2 * KU * step;
  const uint32_t ring = smem_u32(s_dyn) + threadIdx.x * CB;
  const Shared sh(s_dyn + (VEC == 1 ? 0 : kStages * 2 * KU * CB / 16 * blockDim.x), deal.tok * slots, half);
  const int rows = MODE ? p.H + 2 * p.Hkv : p.H + p.Hkv;
  const Mine me(p, deal, rows);
  const int gl = threadIdx.x % ln;
  const bool is_q = me.r < p.H, is_v = MODE && me.r >= p.H + p.Hkv;
  const int h = is_q ? me.r : me.r - p.H - (is_v ? p.Hkv : 0);  // head of q, k or v
  int oa[KU], ob[KU], have = 0;
#pragma unroll
  for (int k = 0; k < KU; ++k) {
    unit_at<VEC, HALF>(gl + k * ln, ru, half, oa[k], ob[k]);
    if (me.on && gl + k * ln < U) have = k + 1;
  }
  const int64_t in_token = is_q ? p.q_token : is_v ? p.v_token : p.k_token;
  const int64_t in_step = in_token * deal.per_round;
  const int64_t out_token = is_q ? p.q_out_token : p.k_out_token;
  int64_t t = me.begin + me.tr, ahead = t;  // tokens of the round, and of the fetch
  const T* src = static_cast<const T*>(is_q ? p.q : is_v ? p.v : p.k) + t * in_token +
                 h * (is_q ? p.q_head : is_v ? static_cast<int64_t>(p.d) : p.k_head);
  T* dst = MODE && !is_q ? nullptr
                         : static_cast<T*>(is_q ? p.q_out : p.k_out) + t * out_token +
                               h * (is_q ? p.q_out_head : p.k_out_head);
  uint32_t in = 0, out = 0;  // stages of the ring
  auto fetch = [&] {
    if (ahead < me.end) X::fetch(ring + in, step, src, oa, ob, have);
    copy_commit();
    ahead += deal.per_round;
    src += in_step;
    in = in == (kStages - 1) * stage ? 0 : in + stage;
  };
  if constexpr (VEC > 1) {  // under way while the angles are made
#pragma unroll
    for (int i = 0; i < kStages - 1; ++i) fetch();
  }
  Ahead first;
  first.load(p, me.begin, static_cast<int>(min(static_cast<int64_t>(deal.tok), me.end - me.begin)));
  uint64_t wA[N2], wB[N2];
  if (p.norm && !is_v)
    weights_of<DT, VEC, KU, HALF>(p, is_q ? p.q_weight : p.k_weight, oa, ob, have, wA, wB);
  // warps whose groups are all v's form no norm, those with none of k or v no bytes
  const bool normed = p.norm && __any_sync(kAll, !is_v);
  const bool cached = MODE == 2 && __any_sync(kAll, me.on && !is_q);
  const float inv_d = 1.f / p.d;
  fill_fixed<VEC>(p, sh, first, deal.tok, slots);
  for (int64_t t0 = me.begin; t0 < me.end; t0 += deal.tok) {
    const int nt = static_cast<int>(min(static_cast<int64_t>(deal.tok), me.end - t0));
    if constexpr (MODE) {
      sequences_of(p.cu, p.B, static_cast<int>(p.T), p.status, t0, nt, s_seq);
      if (threadIdx.x < nt) {
        const int64_t tt = t0 + threadIdx.x;
        const int b = s_seq[threadIdx.x];
        int64_t slot = -2, pos = 0;
        if (b != kNobody) {
          const int64_t at = static_cast<int64_t>(p.ctx[b]) + (tt - p.cu[b]);
          const int64_t lp = at / p.page_size;
          const bool in_table = p.ctx[b] >= 0 && lp < p.max_pages;
          const int phys =
              in_table ? p.block_table[static_cast<size_t>(b) * p.max_pages + lp] : -1;
          slot = -1;
          if (phys < 0 || phys >= p.num_pages)
            atomicOr(p.status, FA_DEV_BAD_PAGE);
          else
            slot = static_cast<int64_t>(phys) * p.Hkv * p.page_size + (at - lp * p.page_size);
          pos = at;
        }
        s_dst[threadIdx.x] = slot;  // -2: nobody's token, nothing is written; -1: no slot, q alone is
        if (!p.pos) s_pos[0][threadIdx.x] = pos;
      }
    }
    if (p.pos) fill_positions(p, s_pos, t0, nt, t0 == me.begin, first);
    __syncthreads();  // also: the last batch's sines have been read
    fill_angles<VEC>(p, nt, sh, slots, p.inverse != 0, [&](int a, int i) { return s_pos[a][i]; });
    __syncthreads();
    // every lane goes round alike; the last round may have no token for it
    for (int tk = me.tr; tk - me.tr < nt; tk += deal.per_round) {
      const bool live = me.on && tk < nt;
      X x;
      if constexpr (VEC > 1) {
        copy_wait<kStages - 2>();
        x.take(ring + out, step, have);
        out = out == (kStages - 1) * stage ? 0 : out + stage;
        fetch();
      } else {
        x.clear();
        if (live) x.load(src, oa, ob, have);
        src += in_step;
      }
      uint64_t A[N2], B[N2];
      x.widen(A, B);
      if (normed) {  // (elements that the row does not have are zeros)
        uint64_t sa = 0, sb = 0;
#pragma unroll
        for (int i = 0; i < N2; ++i) {
          sa = f2_fma(A[i], A[i], sa);
          sb = f2_fma(B[i], B[i], sb);
        }
        const float ss = sum_lanes(f2_sum(f2_add(sa, sb)), ln);
        if (!is_v) {
          const float rr = rsqrtf(fmaf(ss, inv_d, p.eps));
          const uint64_t rr2 = f2(rr, rr);
          // x r first: w x alone may leave FP32, and an infinitely long row (r = 0) is to become zeros
#pragma unroll
          for (int i = 0; i < N2; ++i) {
            A[i] = f2_mul(f2_mul(A[i], rr2), wA[i]);
            B[i] = f2_mul(f2_mul(B[i], rr2), wB[i]);
          }
        }
      }
      if (!is_v && live) {
        const uint64_t minus = f2(-1.f, -1.f);
        uint64_t nB[N2];
#pragma unroll
        for (int i = 0; i < N2; ++i) nB[i] = f2_mul(B[i], minus);
        turn<VEC, N2, RAGGED>(A, B, nB, sh.cs + tk * slots, gl, ln, ru, half);
      }
      const int64_t slot = MODE && live ? s_dst[tk] : 0;
      if (MODE == 2 && cached) {  // every group of the warp takes part in the shuffles
        float big = 0.f;
#pragma unroll
        for (int i = 0; i < N2; ++i) {
          float u, v;
          f2_split(A[i], u, v);
          big = max3_abs_nan(big, u, v);
          f2_split(B[i], u, v);
          big = max3_abs_nan(big, u, v);
        }
        uint32_t bits = __float_as_uint(big);  // (a NaN's are above an infinity's)
        for (int o = ln / 2; o > 0; o /= 2) bits = max(bits, __shfl_xor_sync(kAll, bits, o));
        if (live && !is_q && slot >= 0) {
          const int byte = power_byte(bits);
          const float up = byte == 255 ? 0.f : up_of(byte);
          const int64_t row = slot + static_cast<int64_t>(h) * p.page_size;
          uint8_t* const to = static_cast<uint8_t*>(is_v ? p.v_pages : p.k_pages) + row * p.d;
          if (gl == 0) (is_v ? p.v_scales : p.k_scales)[row] = static_cast<uint8_t>(byte);
          Chunk<uint8_t, VEC> oc[2 * KU];
#pragma unroll
          for (int i = 0; i < N2; ++i) {
            float a0, a1, b0, b1;
            f2_split(f2_mul(A[i], f2(up, up)), a0, a1);
            f2_split(f2_mul(B[i], f2(up, up)), b0, b1);
            // neighbours in the row: of the chunk, or of the pair
            uint32_t lo = HALF || VEC == 1 ? cvt_e4m3x2(a0, a1) : cvt_e4m3x2(a0, b0);
            uint32_t hi = HALF || VEC == 1 ? cvt_e4m3x2(b0, b1) : cvt_e4m3x2(a1, b1);
            if (byte == 255) lo = hi = 0;
            const int k = 2 * i / VEC, e = 2 * i % VEC;
            if (VEC == 1) {
              oc[2 * (2 * i)].e[0] = static_cast<uint8_t>(lo);
              oc[2 * (2 * i + 1)].e[0] = static_cast<uint8_t>(lo >> 8);
              oc[2 * (2 * i) + 1].e[0] = static_cast<uint8_t>(hi);
              oc[2 * (2 * i + 1) + 1].e[0] = static_cast<uint8_t>(hi >> 8);
            } else if (HALF) {
              oc[2 * k].e[e] = static_cast<uint8_t>(lo);
              oc[2 * k].e[(e + 1) % VEC] = static_cast<uint8_t>(lo >> 8);
              oc[2 * k + 1].e[e] = static_cast<uint8_t>(hi);
              oc[2 * k + 1].e[(e + 1) % VEC] = static_cast<uint8_t>(hi >> 8);
            } else {
              Chunk<uint8_t, VEC>& o = oc[2 * k + (2 * e >= VEC ? 1 : 0)];
              o.e[(2 * e) % VEC] = static_cast<uint8_t>(lo);
              o.e[(2 * e + 1) % VEC] = static_cast<uint8_t>(lo >> 8);
              o.e[(2 * e + 2) % VEC] = static_cast<uint8_t>(hi);
              o.e[(2 * e + 3) % VEC] = static_cast<uint8_t>(hi >> 8);
            }
          }
#pragma unroll
          for (int k = 0; k < KU; ++k)
            if (k < have) {
              *reinterpret_cast<Chunk<uint8_t, VEC>*>(to + oa[k]) = oc[2 * k];
              *reinterpret_cast<Chunk<uint8_t, VEC>*>(to + ob[k]) = oc[2 * k + 1];
            }
        }
      }
      T* const to = dst;
      dst += out_token * deal.per_round;
      if (!live) continue;
      if (MODE == 0 || is_q) {
        if (MODE == 0 || slot != -2) X::store(to, oa, ob, have, A, B);
      } else if (MODE == 1 && slot >= 0) {
        X::store(static_cast<T*>(is_v ? p.v_pages : p.k_pages) +
                     (slot + static_cast<int64_t>(h) * p.page_size) * p.d,
                 oa, ob, have, A, B);
      }
    }
  }
}

// The gradient. A thread has the same elements of one head of every token, so the weight's gradient
// adds up in its registers; they meet once at the end, per CTA, in a fixed order, and
// norm_rope_sum_kernel adds the CTAs in theirs: the same bits on every run of the same sizes.
template <int DT, int VEC, int KU, bool HALF, bool RAGGED>
__global__ void __launch_bounds__(kMostThreads, VEC == 1 ? 1 : 2)
    norm_rope_bwd_kernel(const __grid_constant__ NormRopeParams p, const Deal deal) {
  using T = typename Elem<DT>::T;
  using X = Part<DT, VEC, KU, HALF>;
  constexpr int N2 = X::N2, kGradStages = grad_stages(KU * VEC * sizeof(T) / 16);
  extern __shared__ float4 s_dyn[];
  __shared__ int64_t s_pos[FA_MAX_AXES][kTokMax];
  const int half = p.rot / 2, ru = (half + VEC - 1) / VEC, slots = ru * VEC;
  const int U = p.d / (2 * VEC), ln = deal.ln;
  constexpr int CB = sizeof(typename X::C);
  const uint32_t step = blockDim.x * CB, stage = 4 * KU * step;
  const uint32_t ring = smem_u32(s_dyn) + threadIdx.x * CB;
  const Shared sh(s_dyn + (VEC == 1 ? 0 : kGradStages * 4 * KU * CB / 16 * blockDim.x),
                  deal.tok * slots, half);
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");  // the summing kernel may come up
  const Mine me(p, deal, p.H + p.Hkv);
  const int gl = threadIdx.x % ln;
  const bool is_k = me.r >= p.H;
  const int h = is_k ? me.r - p.H : me.r;
  int oa[KU], ob[KU], have = 0;
#pragma unroll
  for (int k = 0; k < KU; ++k) {
    unit_at<VEC, HALF>(gl + k * ln, ru, half, oa[k], ob[k]);
    if (me.on && gl + k * ln < U) have = k + 1;
  }
  const int64_t x_token = is_k ? p.k_token : p.q_token, y_token = is_k ? p.dyk_token : p.dyq_token;
  const int64_t d_token = is_k ? p.k_out_token : p.q_out_token;
  int64_t ahead = me.begin + me.tr;
  const T* px = static_cast<const T*>(is_k ? p.k : p.q) + ahead * x_token +
                h * (is_k ? p.k_head : p.q_head);
  const T* py = static_cast<const T*>(is_k ? p.dyk : p.dyq) + ahead * y_token +
                h * (is_k ? p.dyk_head : p.dyq_head);
  T* dst = static_cast<T*>(is_k ? p.k_out : p.q_out) + ahead * d_token +
           h * (is_k ? p.k_out_head : p.q_out_head);
  uint32_t in = 0, out = 0;  // stages of the ring
  auto fetch = [&] {
    if (ahead < me.end) {
      X::fetch(ring + in, step, px, oa, ob, have);
      X::fetch(ring + in + 2 * KU * step, step, py, oa, ob, have);
    }
    copy_commit();
    ahead += deal.per_round;
    px += x_token * deal.per_round;
    py += y_token * deal.per_round;
    in = in == (kGradStages - 1) * stage ? 0 : in + stage;
  };
  if constexpr (VEC > 1) {
#pragma unroll
    for (int i = 0; i < kGradStages - 1; ++i) fetch();
  }
  Ahead first;
  first.load(p, me.begin, static_cast<int>(min(static_cast<int64_t>(deal.tok), me.end - me.begin)));
  uint64_t wA[N2], wB[N2], da[N2], db[N2];  // the weight and its gradient
  weights_of<DT, VEC, KU, HALF>(p, is_k ? p.k_weight : p.q_weight, oa, ob, have, wA, wB);
#pragma unroll
  for (int i = 0; i < N2; ++i) da[i] = db[i] = 0;
  const float inv_d = 1.f / p.d;
  fill_fixed<VEC>(p, sh, first, deal.tok, slots);
  for (int64_t t0 = me.begin; t0 < me.end; t0 += deal.tok) {
    const int nt = static_cast<int>(min(static_cast<int64_t>(deal.tok), me.end - t0));
    fill_positions(p, s_pos, t0, nt, t0 == me.begin, first);
    __syncthreads();  // also: the last batch's sines have been read
    fill_angles<VEC>(p, nt, sh, slots, true, [&](int a, int i) { return s_pos[a][i]; });
    __syncthreads();
    for (int tk = me.tr; tk - me.tr < nt; tk += deal.per_round) {
      const bool live = me.on && tk < nt;
      X x, dy;
      if constexpr (VEC > 1) {
        copy_wait<kGradStages - 2>();
        x.take(ring + out, step, have);
        dy.take(ring + out + 2 * KU * step, step, have);
        out = out == (kGradStages - 1) * stage ? 0 : out + stage;
        fetch();
      } else {
        x.clear();
        dy.clear();
        if (live) {
          x.load(px, oa, ob, have);
          dy.load(py, oa, ob, have);
        }
        px += x_token * deal.per_round;
        py += y_token * deal.per_round;
      }
      uint64_t A[N2], B[N2], gA[N2], gB[N2];
      dy.widen(gA, gB);
      if (live) {
        const uint64_t minus = f2(-1.f, -1.f);
        uint64_t nB[N2];
#pragma unroll
        for (int i = 0; i < N2; ++i) nB[i] = f2_mul(gB[i], minus);
        turn<VEC, N2, RAGGED>(gA, gB, nB, sh.cs + tk * slots, gl, ln, ru, half);
      }
      x.widen(A, B);
      uint64_t ss2 = 0, sg2 = 0;
#pragma unroll
      for (int i = 0; i < N2; ++i) {
        ss2 = f2_fma(A[i], A[i], f2_fma(B[i], B[i], ss2));
        sg2 = f2_fma(f2_mul(gA[i], wA[i]), A[i], f2_fma(f2_mul(gB[i], wB[i]), B[i], sg2));
      }
      const float ss = sum_lanes(f2_sum(ss2), ln), sg = sum_lanes(f2_sum(sg2), ln);
      T* const to = dst;
      dst += d_token * deal.per_round;
      if (!live) continue;
      // r x (sum) first: r^3 alone leaves FP32 for rows below 1e-13. An infinitely long row (r = 0) has no
      // gradient, though its sum may be infinite.
      const float rr = rsqrtf(fmaf(ss, inv_d, p.eps));
      const float c = rr == 0.f ? 0.f : -(rr * (sg * inv_d)) * rr * rr;
      const uint64_t rr2 = f2(rr, rr), c2 = f2(c, c);
#pragma unroll
      for (int i = 0; i < N2; ++i) {
        const uint64_t ga = f2_mul(gA[i], rr2), gb = f2_mul(gB[i], rr2);
        da[i] = f2_fma(ga, A[i], da[i]);
        db[i] = f2_fma(gb, B[i], db[i]);
        A[i] = f2_fma(A[i], c2, f2_mul(ga, wA[i]));
        B[i] = f2_fma(B[i], c2, f2_mul(gb, wB[i]));
      }
      X::store(to, oa, ob, have, A, B);
    }
  }
  if (!p.part) return;
  // the CTA's groups, first those of q's heads and then those of k's, one after the other
  copy_wait<0>();
  __syncthreads();  // the ring becomes [groups][d]
  float* const s_dw = reinterpret_cast<float*>(s_dyn);
#pragma unroll
  for (int i = 0; i < N2; ++i) {
    float v[4];  // A, A of the next pair, B, B
    f2_split(da[i], v[0], v[1]);
    f2_split(db[i], v[2], v[3]);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int n = 2 * i + j % 2, k = n / VEC, e = n % VEC;
      const int at = HALF || VEC == 1 ? (j < 2 ? oa[k] : ob[k]) + e : oa[k] + 2 * e + j / 2;
      if (k < have) s_dw[threadIdx.x / ln * p.d + at] = v[j];
    }
  }
  __syncthreads();
  const size_t cta = static_cast<size_t>(blockIdx.y) * gridDim.x + blockIdx.x;
  for (int i = threadIdx.x; i < 2 * p.d; i += blockDim.x) {
    const int kd = i >= p.d ? 1 : 0, c = i - kd * p.d;
    const int first = blockIdx.y * deal.heads;
    const int from = kd ? max(0, p.H - first) : 0;
    const int to = kd ? min(deal.heads, p.H + p.Hkv - first) : min(deal.heads, p.H - first);
    float s = 0.f;
    for (int t = 0; t < deal.per_round; ++t) {
      const float* const x = s_dw + t * deal.heads * p.d + c;
#pragma unroll 8
      for (int r = from; r < to; ++r) s += x[r * p.d];
    }
    p.part[(cta * 2 + kd) * p.d + c] = s;
  }
}

// Column c of the CTAs' partial sums [ctas][2][d]: 32 columns and 32 shares of the CTAs per CTA;
// blockIdx.y picks the weight.
__global__ void __launch_bounds__(1024)
    norm_rope_sum_kernel(const float* part, int ctas, int d, float* dq_weight, float* dk_weight) {
  __shared__ float s[32][33];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  float* const out = blockIdx.y ? dk_weight : dq_weight;
  if (!out) return;
  const int lane = threadIdx.x % 32, share = threadIdx.x / 32, c = blockIdx.x * 32 + lane;
  const float* const mine = part + static_cast<size_t>(blockIdx.y) * d + c;
  float x[4] = {0.f, 0.f, 0.f, 0.f};
  if (c < d)
    for (int i = share; i < ctas; i += 128) {
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (i + 32 * j < ctas) x[j] += mine[static_cast<size_t>(i + 32 * j) * 2 * d];
    }
  s[share][lane] = (x[0] + x[1]) + (x[2] + x[3]);
  __syncthreads();
  float y = s[lane][share];  // lane: share; share: column
#pragma unroll
  for (int o = 16; o > 0; o /= 2) y += __shfl_xor_sync(kAll, y, o);
  const int col = blockIdx.x * 32 + share;
  if (lane == 0 && col < d) out[col] = y;
}

// Cached rows back as packed 16-bit ones: a CTA takes `tok` tokens, eight or four lanes a row of K
// or V (16 elements each), whose 128 or 64 bytes are one access.
constexpr int kReadTok = 16;
template <bool BF16>
__global__ void __launch_bounds__(kRopeThreads)
    kv_read_kernel(const __grid_constant__ KvReadParams p, int tok) {
  __shared__ int64_t s_src[kReadTok];
  __shared__ int s_seq[kReadTok];
  const int64_t t0 = static_cast<int64_t>(blockIdx.x) * tok;
  const int nt = static_cast<int>(min(static_cast<int64_t>(tok), p.T - t0));
  sequences_of(p.cu, p.B, static_cast<int>(p.T), p.status, t0, nt, s_seq);
  if (threadIdx.x < nt) {
    const int b = s_seq[threadIdx.x];
    int64_t src = -2;
    if (b != kNobody) {
      const int64_t at = static_cast<int64_t>(p.starts[b]) + (t0 + threadIdx.x - p.cu[b]);
      const int64_t lp = at / p.page_size;
      const bool in = p.starts[b] >= 0 && lp < p.max_pages;
      const int phys = in ? p.block_table[static_cast<size_t>(b) * p.max_pages + lp] : -1;
      src = -1;
      if (phys < 0 || phys >= p.num_pages)
        atomicOr(p.status, FA_DEV_BAD_PAGE);
      else
        src = static_cast<int64_t>(phys) * p.Hkv * p.page_size + (at - lp * p.page_size);
    }
    s_src[threadIdx.x] = src;  // -2: nobody's row, left as it was; -1: no slot, zeros
  }
  __syncthreads();
  const int per = p.d / 16, rows = 2 * p.Hkv, total = nt * rows * per;
  for (int j = threadIdx.x; j < total; j += kRopeThreads) {
    const int c = j % per, x = j / per, r = x % rows, tk = x / rows;
    const int64_t src = s_src[tk];
    if (src == -2) continue;
    const bool is_v = r >= p.Hkv;
    const int h = is_v ? r - p.Hkv : r;
    uint4 raw = make_uint4(0, 0, 0, 0);
    float s = 0.f;
    if (src >= 0) {
      const int64_t row = src + static_cast<int64_t>(h) * p.page_size;
      raw = *reinterpret_cast<const uint4*>(
          static_cast<const uint8_t*>(is_v ? p.v_pages : p.k_pages) + row * p.d + 16 * c);
      s = power_of((is_v ? p.v_scales : p.k_scales)[row]);
    }
    uint32_t out[8];
    const uint32_t in[4] = {raw.x, raw.y, raw.z, raw.w};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float2 f = e4m3x2_to_f32(in[i / 2] >> (16 * (i % 2)));
      out[i] = BF16 ? cvt_pack_bf16(f.x * s, f.y * s) : cvt_pack_f16(f.x * s, f.y * s);
    }
    uint4* dst = reinterpret_cast<uint4*>(static_cast<uint16_t*>(is_v ? p.v : p.k) +
                                          (t0 + tk) * (is_v ? p.v_token : p.k_token) +
                                          static_cast<int64_t>(h) * p.d + 16 * c);
    dst[0] = make_uint4(out[0], out[1], out[2], out[3]);
    dst[1] = make_uint4(out[4], out[5], out[6], out[7]);
  }
}

// Lanes of a row: a power of two, at most `ku` units to a lane.
int lanes_of(int units, int ku) {
  int ln = 1;
  while (ln * ku < units) ln *= 2;
  return ln;
}

// The deal of `rows` heads of T tokens over as many CTAs as give an SM at most `per_sm` threads, and at
// most `most`, with `ring` bytes of rows on their way per thread.
struct Launch {
  Deal deal;
  dim3 grid;
  int threads, smem;
};
Launch deal_rows(const NormRopeParams& p, int ln, int vec, int rows, int sms, int per_sm, int most,
                 int ring) {
  Launch L;
  Deal& d = L.deal;
  d.ln = ln;
  // all heads of a token side by side, or several equal shares of them; several tokens of few heads
  const int chunks = (rows * ln + kMostThreads - 1) / kMostThreads;
  d.heads = (rows + chunks - 1) / chunks;
  d.per_round = std::max(1, 256 / (d.heads * ln));
  d.per_round = static_cast<int>(std::min<int64_t>({d.per_round, p.T, kTokMax}));
  L.threads = (d.per_round * d.heads * ln + 31) / 32 * 32;
  const int64_t runs = (p.T + d.per_round - 1) / d.per_round;  // rounds of all tokens
  const int ctas = std::min(most, sms * (per_sm / L.threads));
  L.grid = dim3(static_cast<unsigned>(std::min<int64_t>(runs, std::max(1, ctas / chunks))), chunks);
  // the sines of a batch within 12 KB; no more than the CTA's own tokens
  const int64_t own = (p.T + L.grid.x - 1) / L.grid.x;
  const int slots = (p.rot / 2 + vec - 1) / vec * vec;
  int64_t tok = std::min<int64_t>({kTokMax, 12288 / (slots * 8),
                                   (own + d.per_round - 1) / d.per_round * d.per_round});
  d.tok = static_cast<int>(std::max<int64_t>(1, tok / d.per_round)) * d.per_round;
  L.smem = shared_bytes(d.tok * slots, p.rot / 2) + ring * L.threads;
  return L;
}
constexpr int kMostShared = 16384 + kTokMax * 256 * 8;  // beside the ring

// bytes of rows on their way per thread: `parts` halves of a lane's part
template <int DT, int VEC, int KU>
constexpr int ring_bytes(int parts) {
  return VEC == 1 ? 0 : parts * KU * VEC * static_cast<int>(sizeof(typename Elem<DT>::T));
}
// f(half layout, neighbours whose last unit is rotated in part): chunks below 16 bytes are for halves alone,
// and a kernel of its own keeps the rest free of the registers that such units take (the gradient of
// 8191 tokens x 20 heads of 64, half of them rotated: 26.2 us with one kernel, 24.8 so).
template <int DT, int VEC, typename F>
void pick_kernel(const NormRopeParams& p, bool half_style, F f) {
  constexpr bool kWide = VEC * sizeof(typename Elem<DT>::T) == 16;
  if constexpr (VEC == 1 || kWide) {
    if (!half_style) {
      if constexpr (kWide)
        if (p.rot / 2 % VEC) return f(std::false_type{}, std::true_type{});
      return f(std::false_type{}, std::false_type{});
    }
  }
  f(std::true_type{}, std::false_type{});
}
template <int DT, int VEC, int KU, int MODE>
cudaError_t launch_v(const NormRopeParams& p, bool half_style, int sms, cudaStream_t stream) {
  constexpr int ring = ring_bytes<DT, VEC, KU>(kStages * 2);
  constexpr int most = kMostShared + ring * kMostThreads;
  const Launch L = deal_rows(p, lanes_of(p.d / (2 * VEC), KU), VEC, p.H + (MODE ? 2 : 1) * p.Hkv,
                             sms, ctas_per_sm(DT, VEC, MODE) * kMostThreads, INT_MAX, ring);
  void (*k)(NormRopeParams, Deal);
  cudaError_t e;
  pick_kernel<DT, VEC>(p, half_style, [&](auto half, auto ragged) {
    constexpr bool H = decltype(half)::value, R = decltype(ragged)::value;
    k = norm_rope_kernel<DT, VEC, KU, H, R, MODE>;
    e = prepare_kernel<norm_rope_kernel<DT, VEC, KU, H, R, MODE>>(most);
  });
  if (e != cudaSuccess) return e;
  k<<<L.grid, L.threads, L.smem, stream>>>(p, L.deal);
  return cudaGetLastError();
}
template <int DT, int VEC, int KU>
cudaError_t launch_bwd_v(const NormRopeParams& p, bool half_style, int sms, cudaStream_t stream) {
  constexpr int ring = ring_bytes<DT, VEC, KU>(grad_stages(KU * VEC * (DT == FA_F32 ? 2 : 1) / 8) * 4);
  constexpr int most = kMostShared + ring * kMostThreads;
  Launch L = deal_rows(p, lanes_of(p.d / (2 * VEC), KU), VEC, p.H + p.Hkv, sms,
                       (VEC == 1 ? 1 : 2) * kMostThreads, kNormCtas, ring);
  // the weights' gradients of its groups meet in the ring's place
  L.smem = std::max(L.smem, L.deal.per_round * L.deal.heads * p.d * 4);
  void (*k)(NormRopeParams, Deal);
  cudaError_t e;
  pick_kernel<DT, VEC>(p, half_style, [&](auto half, auto ragged) {
    constexpr bool H = decltype(half)::value, R = decltype(ragged)::value;
    k = norm_rope_bwd_kernel<DT, VEC, KU, H, R>;
    e = prepare_kernel<norm_rope_bwd_kernel<DT, VEC, KU, H, R>>(most);
  });
  if (e != cudaSuccess) return e;
  k<<<L.grid, L.threads, L.smem, stream>>>(p, L.deal);
  e = cudaGetLastError();
  if (e != cudaSuccess || !p.part) return e;
  cudaLaunchAttribute early;  // it may come up while the gradient runs, which it then waits for
  early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  early.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((p.d + 31) / 32, 2);
  cfg.blockDim = dim3(1024);
  cfg.stream = stream;
  cfg.attrs = &early;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, norm_rope_sum_kernel, static_cast<const float*>(p.part),
                            static_cast<int>(L.grid.x * L.grid.y), p.d, p.dq_weight, p.dk_weight);
}

// Elements of a chunk, at most 16 bytes: what the rotated halves divide into (neighbours need no such
// thing). Steps and pointers are multiples of 16 bytes; without that, 1.
int chunk_of(const NormRopeParams& p, bool half_style, bool vec, int most) {
  int v = vec && p.d % (2 * most) == 0 ? most : 1;
  while (half_style && v > 1 && (p.rot / 2) % v) v /= 2;
  return v;
}
template <int DT, int MODE>
cudaError_t launch_m(const NormRopeParams& p, bool half_style, bool vec, int sms,
                     cudaStream_t stream) {
  constexpr int most = DT == FA_F32 ? 4 : 8;
  switch (chunk_of(p, half_style, vec, most)) {
    case most: return launch_v<DT, most, 8 / most, MODE>(p, half_style, sms, stream);
    case most / 2: return launch_v<DT, most / 2, 16 / most, MODE>(p, half_style, sms, stream);
    case most / 4: if (most > 4) return launch_v<DT, 2, 4, MODE>(p, half_style, sms, stream);
  }
  return launch_v<DT, 1, 8, MODE>(p, half_style, sms, stream);
}
template <int DT>
cudaError_t launch_bwd_t(const NormRopeParams& p, bool half_style, bool vec, int sms,
                         cudaStream_t stream) {
  constexpr int most = DT == FA_F32 ? 4 : 8;
  switch (chunk_of(p, half_style, vec, most)) {
    case most: return launch_bwd_v<DT, most, 8 / most>(p, half_style, sms, stream);
    case most / 2: return launch_bwd_v<DT, most / 2, 16 / most>(p, half_style, sms, stream);
    case most / 4: if (most > 4) return launch_bwd_v<DT, 2, 4>(p, half_style, sms, stream);
  }
  return launch_bwd_v<DT, 1, 8>(p, half_style, sms, stream);
}

}  // namespace

cudaError_t launch_norm_rope(const NormRopeParams& p, int dtype, bool half_style, bool vec,
                             int sms, cudaStream_t stream) {
  if (dtype == FA_F32) return launch_m<FA_F32, 0>(p, half_style, vec, sms, stream);
  if (dtype == FA_BF16) return launch_m<FA_BF16, 0>(p, half_style, vec, sms, stream);
  return launch_m<FA_F16, 0>(p, half_style, vec, sms, stream);
}

cudaError_t launch_norm_rope_bwd(const NormRopeParams& p, int dtype, bool half_style, bool vec,
                                 int sms, cudaStream_t stream) {
  if (dtype == FA_F32) return launch_bwd_t<FA_F32>(p, half_style, vec, sms, stream);
  if (dtype == FA_BF16) return launch_bwd_t<FA_BF16>(p, half_style, vec, sms, stream);
  return launch_bwd_t<FA_F16>(p, half_style, vec, sms, stream);
}

cudaError_t launch_norm_rope_append(const NormRopeParams& p, int dtype, bool half_style, bool vec,
                                    int sms, cudaStream_t stream) {
  const bool q8 = p.k_scales != nullptr;
  if (dtype == FA_BF16)
    return q8 ? launch_m<FA_BF16, 2>(p, half_style, vec, sms, stream)
              : launch_m<FA_BF16, 1>(p, half_style, vec, sms, stream);
  return q8 ? launch_m<FA_F16, 2>(p, half_style, vec, sms, stream)
            : launch_m<FA_F16, 1>(p, half_style, vec, sms, stream);
}

cudaError_t launch_kv_read(const KvReadParams& p, bool bf16, int sms, cudaStream_t stream) {
  const int tok = p.T >= 64LL * sms ? 16 : p.T >= 8LL * sms ? 4 : 1;
  const int64_t grid = (p.T + tok - 1) / tok;
  if (bf16)
    kv_read_kernel<true><<<static_cast<unsigned>(grid), kRopeThreads, 0, stream>>>(p, tok);
  else
    kv_read_kernel<false><<<static_cast<unsigned>(grid), kRopeThreads, 0, stream>>>(p, tok);
  return cudaGetLastError();
}

}  // namespace fa
