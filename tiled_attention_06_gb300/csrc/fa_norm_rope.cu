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
// HBM does in bulk and latency in a decode step. A row is spread over LN neighbouring lanes, 16
// elements to a lane, whose sums meet in log2(LN) shuffles; a group of lanes keeps to one token
// and takes its heads one after the other, so the sines, cosines and the weight stay in registers,
// and the next head's load is under way while one is worked on.
#include <algorithm>
#include <cstdint>

#include "fa_ptx.cuh"
#include "fa_rope.cuh"

namespace fa {
namespace {

constexpr int kTokMax = 32;  // tokens of a CTA at most
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
// A CTA's shared memory: sines and cosines of its tokens, the frequencies, the weights of q and k,
// the pairs' axes. For VEC > 1 the cosines and sines (the weights of A and B) of two pairs are 16
// bytes, neighbouring units next to each other, so that neighbouring lanes read neighbouring 16 bytes.
struct Shared {
  float2* cs;
  uint64_t* freq;
  float* w;
  uint8_t* axis;
  __device__ __forceinline__ Shared(float4* base, int tok, int half, int d) {
    cs = reinterpret_cast<float2*>(base);
    w = reinterpret_cast<float*>(cs + static_cast<size_t>((tok * half + 1) & ~1));
    freq = reinterpret_cast<uint64_t*>(w + static_cast<size_t>((2 * d + 3) & ~3));
    axis = reinterpret_cast<uint8_t*>(freq + half);
  }
};
size_t shared_bytes(int tok, int half, int d) {
  return static_cast<size_t>((tok * half + 1) & ~1) * 8 + static_cast<size_t>((2 * d + 3) & ~3) * 4 +
         static_cast<size_t>(half) * 9;
}
// Rows on their way: every thread copies its own 16-byte chunks of the rows to come to shared memory
// (cp.async, three rounds ahead and on into the next batch) and reads them back itself, so nothing waits
// for anyone else. In registers a row ahead is what there is room for: 32 KB per SM on their way,
// 73 us where this takes 5x, 152 us for the gradient's 9x.
constexpr int kStages = 4;
template <int VEC>
__host__ __device__ constexpr int ring_bytes(int chunks) {  // chunks of 16 bytes, per thread and round
  return VEC == 1 ? 0 : kStages * chunks * kRopeThreads * 16;
}
__device__ __forceinline__ void copy_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copy_commit() {
  asm volatile("cp.async.commit_group;" ::: "memory");
}
template <int N>
__device__ __forceinline__ void copy_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ float weight_at(const void* w, int f32, int dt, int i) {
  if (!w) return 1.f;
  if (f32) return static_cast<const float*>(w)[i];
  const uint16_t x = static_cast<const uint16_t*>(w)[i];
  return dt == FA_BF16 ? Elem<FA_BF16>::get(x) : Elem<FA_F16>::get(x);
}

// Where the first of pair e of unit u's two numbers lies (the second is two behind it for VEC > 1,
// one for VEC = 1), `units` of them in all: [e / 2][u][A_e A_{e+1} B_e B_{e+1}], or [u][A B].
template <int VEC>
__device__ __forceinline__ int pair_at(int u, int e, int units) {
  return VEC == 1 ? 2 * u : ((e / 2) * units + u) * 4 + e % 2;
}

// Frequencies, axes and weights: the part that does not depend on the tokens.
template <int DT, int VEC, bool HALF>
__device__ __forceinline__ void fill_fixed(const NormRopeParams& p, const Shared& sh) {
  const int half = p.rot / 2, ru = half / VEC, U = p.d / (2 * VEC);
  for (int i = threadIdx.x; i < half; i += kRopeThreads) {
    sh.freq[i] = turns_q64(p.freqs[i]);
    int a = p.pair_axis ? p.pair_axis[i] : 0;
    if (a < 0 || a >= p.axes) {
      if (blockIdx.x == 0) atomicOr(p.status, FA_DEV_BAD_PAGE);
      a = 0;
    }
    sh.axis[i] = static_cast<uint8_t>(a);
  }
  if (!p.norm) return;
  for (int i = threadIdx.x; i < 2 * U * VEC; i += kRopeThreads) {
    const int e = i % VEC, q = i / VEC, kind = q >= U ? 1 : 0, u = q - kind * U;
    const void* const w = kind ? p.k_weight : p.q_weight;
    int oa, ob;
    unit_at<VEC, HALF>(u, ru, half, oa, ob);
    float* const at = sh.w + kind * p.d + pair_at<VEC>(u, e, U);
    at[0] = weight_at(w, p.w_f32, DT, HALF || VEC == 1 ? oa + e : oa + 2 * e);
    at[VEC == 1 ? 1 : 2] = weight_at(w, p.w_f32, DT, HALF || VEC == 1 ? ob + e : oa + 2 * e + 1);
  }
}
// Sines and cosines of nt tokens; pos(axis, token) in 64 bits.
template <int VEC, typename Pos>
__device__ __forceinline__ void fill_angles(const NormRopeParams& p, int nt, const Shared& sh,
                                            bool inverse, Pos pos) {
  const int half = p.rot / 2, ru = half / VEC;
  const int dt = kRopeThreads / half, df = kRopeThreads % half;
  int tk = threadIdx.x / half, f = threadIdx.x % half;
  while (tk < nt) {
    const int64_t at = pos(sh.axis[f], tk);
    const uint64_t phase = static_cast<uint64_t>(inverse ? -at : at) * sh.freq[f];
    float s, c;  // the phase as a signed fraction of a turn: half turns in [-1, 1]
    sincospif(static_cast<float>(static_cast<int64_t>(phase)) * 1.08420217248550443e-19f, &s, &c);
    float* const to = reinterpret_cast<float*>(sh.cs + tk * half) + pair_at<VEC>(f / VEC, f % VEC, ru);
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

__device__ __forceinline__ uint64_t f2_mul(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ uint64_t f2_neg(uint64_t a) { return a ^ 0x8000000080000000ull; }
__device__ __forceinline__ float f2_sum(uint64_t a) {
  float x, y;
  f2_split(a, x, y);
  return x + y;
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
  // the same by way of shared memory: chunk c of the thread at c * kRopeThreads * 16
  static __device__ __forceinline__ void fetch(uint32_t at, const T* src, const int* oa,
                                               const int* ob, int have) {
#pragma unroll
    for (int k = 0; k < KU; ++k)
      if (k < have) {
        copy_async16(at + (2 * k) * (kRopeThreads * 16), src + oa[k]);
        copy_async16(at + (2 * k + 1) * (kRopeThreads * 16), src + ob[k]);
      }
  }
  __device__ __forceinline__ void take(const uint8_t* at, int have) {
    clear();
#pragma unroll
    for (int k = 0; k < KU; ++k)
      if (k < have) {
        a[k] = *reinterpret_cast<const C*>(at + (2 * k) * (kRopeThreads * 16));
        b[k] = *reinterpret_cast<const C*>(at + (2 * k + 1) * (kRopeThreads * 16));
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

// The two numbers of two pairs, (A_e, A_{e+1}) and (B_e, B_{e+1}), for the lane's packed pair i; its
// units are u0, u0 + ln, ... A unit that the row does not have reads the last one's.
template <int VEC>
__device__ __forceinline__ void pairs_of(const float* at, int i, int u0, int ln, int units,
                                         uint64_t& A, uint64_t& B) {
  if constexpr (VEC == 1) {
    const float2 x = *reinterpret_cast<const float2*>(at + 2 * min(u0 + 2 * i * ln, units - 1));
    const float2 y = *reinterpret_cast<const float2*>(at + 2 * min(u0 + (2 * i + 1) * ln, units - 1));
    A = f2(x.x, y.x);
    B = f2(x.y, y.y);
  } else {
    const int u = min(u0 + (2 * i / VEC) * ln, units - 1);
    const ulonglong2 x =
        *reinterpret_cast<const ulonglong2*>(at + pair_at<VEC>(u, 2 * i % VEC, units));
    A = x.x;
    B = x.y;
  }
}
// The rotation of a lane's pairs; those behind the rotated part stay.
template <int VEC, int N2>
__device__ __forceinline__ void turn(uint64_t* A, uint64_t* B, const float2* cs, int u0, int ln,
                                     int ru) {
#pragma unroll
  for (int i = 0; i < N2; ++i) {
    uint64_t c, s;
    pairs_of<VEC>(reinterpret_cast<const float*>(cs), i, u0, ln, ru, c, s);
    if (VEC == 1) {  // two units, of which the rotated part may end with the first
      const bool in0 = u0 + 2 * i * ln < ru, in1 = u0 + (2 * i + 1) * ln < ru;
      const uint64_t lo = 0xffffffffull, one = 0x3f800000ull;
      if (!in0) c = (c & ~lo) | one, s &= ~lo;
      if (!in1) c = (c & lo) | one << 32, s &= lo;
    } else if (u0 + (2 * i / VEC) * ln >= ru) {
      continue;
    }
    const uint64_t a = A[i], b = B[i];
    A[i] = f2_fma(a, c, f2_mul(b, f2_neg(s)));
    B[i] = f2_fma(b, c, f2_mul(a, s));
  }
}
__device__ __forceinline__ float sum_lanes(float x, int ln) {
  for (int o = ln / 2; o > 0; o /= 2) x += __shfl_xor_sync(kAll, x, o);
  return x;
}

// The walk of a group of lanes over the rows of the CTA's batches of tokens, (token, head) with the
// heads first: rows g, g + groups, ... of a batch, and so on in the next one. Every group goes the same
// number of rounds in a batch, in the last of which it may have no row.
struct RowWalk {
  int64_t t0;  // first token of the batch
  int tk, r, left;  // token of the batch, row of it, rows of the batch from this round on
  __device__ __forceinline__ int tokens(const NormRopeParams& p, int tok) const {
    return static_cast<int>(max(static_cast<int64_t>(0), min(static_cast<int64_t>(tok), p.T - t0)));
  }
};
struct RowSteps {
  int g, groups, rows, tok, dt, dr;
  int64_t step;  // tokens between the CTA's batches
  __device__ __forceinline__ RowSteps(int ln, int rows, int tok, int64_t step)
      : g(threadIdx.x / ln),
        groups(kRopeThreads / ln),
        rows(rows),
        tok(tok),
        dt(groups / rows),
        dr(groups % rows),
        step(step) {}
  __device__ __forceinline__ void start(RowWalk& w, const NormRopeParams& p, int64_t t0) const {
    w.t0 = t0;
    w.tk = g / rows;
    w.r = g - w.tk * rows;
    w.left = w.tokens(p, tok) * rows;
  }
  // to the next round of the batch; false at its end
  __device__ __forceinline__ bool next(RowWalk& w) const {
    w.tk += dt;
    w.r += dr;
    if (w.r >= rows) {
      w.r -= rows;
      ++w.tk;
    }
    w.left -= groups;
    return w.left > 0;
  }
};

// Rows r of a token: H of q, Hkv of k and, when appending, Hkv of v. MODE 0: y to q_out and k_out;
// 1 and 2: q to q_out, k and v to the cache's slot of the token, in 16 and in 8 bits. Persistent, every
// grid'th batch of tokens: what comes before the first row (a dozen integer divisions, frequencies,
// weights) was 45 % of all instructions with a CTA per batch of three tokens (91 us, now 6x).
template <int DT, int VEC, int KU, bool HALF, int MODE>
__global__ void __launch_bounds__(kRopeThreads, 4)
    norm_rope_kernel(const __grid_constant__ NormRopeParams p, int tok, int ln) {
  using T = typename Elem<DT>::T;
  using X = Part<DT, VEC, KU, HALF>;
  constexpr int N2 = X::N2;
  extern __shared__ float4 s_dyn[];
  __shared__ int64_t s_dst[kTokMax], s_pos[FA_MAX_AXES][kTokMax];
  __shared__ int s_seq[kTokMax];
  const int half = p.rot / 2, ru = half / VEC, U = p.d / (2 * VEC);
  constexpr int kRing = ring_bytes<VEC>(2 * KU);
  uint8_t* const ring = reinterpret_cast<uint8_t*>(s_dyn) + threadIdx.x * 16;
  const Shared sh(s_dyn + kRing / 16, tok, half, p.d);
  const int gl = threadIdx.x % ln;
  const int rows = MODE ? p.H + 2 * p.Hkv : p.H + p.Hkv;
  int oa[KU], ob[KU], have = 0;
#pragma unroll
  for (int k = 0; k < KU; ++k) {
    unit_at<VEC, HALF>(gl + k * ln, ru, half, oa[k], ob[k]);
    if (gl + k * ln < U) have = k + 1;
  }
  const RowSteps steps(ln, rows, tok, static_cast<int64_t>(gridDim.x) * tok);
  const float inv_d = 1.f / p.d;
  auto row_at = [&](const RowWalk& w) -> const T* {
    const int64_t t = w.t0 + w.tk;
    if (w.r < p.H) return static_cast<const T*>(p.q) + t * p.q_token + w.r * p.q_head;
    if (w.r < p.H + p.Hkv)
      return static_cast<const T*>(p.k) + t * p.k_token + (w.r - p.H) * p.k_head;
    return static_cast<const T*>(p.v) + t * p.v_token +
           static_cast<int64_t>(w.r - p.H - p.Hkv) * p.d;
  };
  RowWalk w, ahead;
  steps.start(ahead, p, static_cast<int64_t>(blockIdx.x) * tok);
  uint32_t in = 0, out = 0;  // rounds fetched and taken
  auto fetch = [&] {
    if (ahead.t0 < p.T) {
      if (ahead.tk < ahead.tokens(p, tok))
        X::fetch(smem_u32(ring) + in % kStages * (kRing / kStages), row_at(ahead), oa, ob, have);
      if (!steps.next(ahead)) steps.start(ahead, p, ahead.t0 + steps.step);
    }
    copy_commit();
    ++in;
  };
  if constexpr (VEC > 1) {
#pragma unroll 1
    for (int i = 0; i < kStages - 1; ++i) fetch();
  }
  bool first = true;
  for (int64_t t0 = static_cast<int64_t>(blockIdx.x) * tok; t0 < p.T; t0 += steps.step) {
    steps.start(w, p, t0);
    const int nt = w.tokens(p, tok);
    if (first) fill_fixed<DT, VEC, HALF>(p, sh);
    first = false;
    if constexpr (MODE) {
      sequences_of(p.cu, p.B, static_cast<int>(p.T), p.status, t0, nt, s_seq);
      if (threadIdx.x < nt) {
        const int64_t tt = t0 + threadIdx.x;
        const int b = s_seq[threadIdx.x];
        int64_t dst = -2, pos = 0;
        if (b != kNobody) {
          const int64_t at = static_cast<int64_t>(p.ctx[b]) + (tt - p.cu[b]);
          const int64_t lp = at / p.page_size;
          const bool in = p.ctx[b] >= 0 && lp < p.max_pages;
          const int phys = in ? p.block_table[static_cast<size_t>(b) * p.max_pages + lp] : -1;
          dst = -1;
          if (phys < 0 || phys >= p.num_pages)
            atomicOr(p.status, FA_DEV_BAD_PAGE);
          else
            dst = static_cast<int64_t>(phys) * p.Hkv * p.page_size + (at - lp * p.page_size);
          pos = at;
        }
        s_dst[threadIdx.x] = dst;  // -2: nobody's token, nothing is written; -1: no slot, q alone is
        if (!p.pos) s_pos[0][threadIdx.x] = pos;
      }
    }
    if (p.pos && threadIdx.x < nt * p.axes) {
      const int a = threadIdx.x / nt, i = threadIdx.x - a * nt;
      s_pos[a][i] = p.pos[a * p.T + t0 + i];
    }
    __syncthreads();  // also: the last batch's sines have been read
    fill_angles<VEC>(p, nt, sh, p.inverse != 0, [&](int a, int i) { return s_pos[a][i]; });
    __syncthreads();

    bool more = true;
    while (more) {  // every lane goes round alike
      const bool live = w.tk < nt, is_v = MODE && w.r >= p.H + p.Hkv;
      const int r = w.r;
      const int64_t t = t0 + w.tk;
      X x;
      if constexpr (VEC > 1) {
        copy_wait<kStages - 2>();
        x.take(ring + out++ % kStages * (kRing / kStages), live ? have : 0);
        fetch();
      } else {
        x.clear();
        if (live) x.load(row_at(w), oa, ob, have);
      }
      uint64_t A[N2], B[N2];
      x.widen(A, B);
      if (p.norm) {  // (elements that the row does not have are zeros)
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
          const float* const wt = sh.w + (r < p.H ? 0 : p.d);
#pragma unroll
          for (int i = 0; i < N2; ++i) {
            uint64_t wa, wb;
            pairs_of<VEC>(wt, i, gl, ln, U, wa, wb);
            A[i] = f2_mul(f2_mul(A[i], rr2), wa);
            B[i] = f2_mul(f2_mul(B[i], rr2), wb);
          }
        }
      }
      if (!is_v && live) turn<VEC, N2>(A, B, sh.cs + w.tk * half, gl, ln, ru);
      const int64_t slot = MODE && live ? s_dst[w.tk] : 0;
      more = steps.next(w);
      if (MODE == 2) {  // every group of the warp takes part in the shuffles
        // the largest magnitude, which passes over NaNs, and zero times everything, which does not
        float big = 0.f;
        uint64_t nan = 0;
#pragma unroll
        for (int i = 0; i < N2; ++i) {
          float u, v;
          f2_split(A[i], u, v);
          big = max3f(big, fabsf(u), fabsf(v));
          f2_split(B[i], u, v);
          big = max3f(big, fabsf(u), fabsf(v));
          nan = f2_fma(A[i], 0, f2_fma(B[i], 0, nan));
        }
        uint32_t bits = f2_sum(nan) == 0.f ? __float_as_uint(big) : 0x7f800000u;
        for (int o = ln / 2; o > 0; o /= 2) bits = max(bits, __shfl_xor_sync(kAll, bits, o));
        if (live && r >= p.H && slot >= 0) {
          const int h = r - p.H - (is_v ? p.Hkv : 0), byte = power_byte(bits);
          const float up = byte == 255 ? 0.f : up_of(byte);
          const int64_t row = slot + static_cast<int64_t>(h) * p.page_size;
          uint8_t* dst = static_cast<uint8_t*>(is_v ? p.v_pages : p.k_pages) + row * p.d;
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
              *reinterpret_cast<Chunk<uint8_t, VEC>*>(dst + oa[k]) = oc[2 * k];
              *reinterpret_cast<Chunk<uint8_t, VEC>*>(dst + ob[k]) = oc[2 * k + 1];
            }
        }
      }
      if (!live || (MODE && (r < p.H ? slot == -2 : MODE == 2 || slot < 0))) continue;
      T* dst;
      if (r < p.H)
        dst = static_cast<T*>(p.q_out) + t * p.q_out_token + r * p.q_out_head;
      else if (MODE == 0)
        dst = static_cast<T*>(p.k_out) + t * p.k_out_token + (r - p.H) * p.k_out_head;
      else
        dst = static_cast<T*>(is_v ? p.v_pages : p.k_pages) +
              (slot + static_cast<int64_t>(r - p.H - (is_v ? p.Hkv : 0)) * p.page_size) * p.d;
      X::store(dst, oa, ob, have, A, B);
    }
  }
}

// The gradient. Persistent, CTAs 0 .. ctas_q - 1 for the heads of q, the others for those of k, each
// over every ctas'th batch of tokens. A thread has the same elements of every row, so the weight's
// gradient adds up in its registers; they meet once at the end, per CTA, in a fixed order, and
// norm_rope_sum_kernel adds the CTAs in theirs: the same bits on every run of the same sizes.
template <int DT, int VEC, int KU, bool HALF>
__global__ void __launch_bounds__(kRopeThreads, VEC == 1 ? 1 : 2)
    norm_rope_bwd_kernel(const __grid_constant__ NormRopeParams p, int tok, int ln, int ctas_q) {
  using T = typename Elem<DT>::T;
  using X = Part<DT, VEC, KU, HALF>;
  constexpr int N2 = X::N2;
  extern __shared__ float4 s_dyn[];
  __shared__ int64_t s_pos[FA_MAX_AXES][kTokMax];
  const int half = p.rot / 2, ru = half / VEC, U = p.d / (2 * VEC);
  constexpr int kRing = ring_bytes<VEC>(4 * KU);
  uint8_t* const ring = reinterpret_cast<uint8_t*>(s_dyn) + threadIdx.x * 16;
  const Shared sh(s_dyn + kRing / 16, tok, half, p.d);
  const int gl = threadIdx.x % ln;
  const bool is_k = static_cast<int>(blockIdx.x) >= ctas_q;
  const int rows = is_k ? p.Hkv : p.H, ctas = is_k ? gridDim.x - ctas_q : ctas_q;
  const T* const px = static_cast<const T*>(is_k ? p.k : p.q);
  const T* const py = static_cast<const T*>(is_k ? p.dyk : p.dyq);
  T* const pd = static_cast<T*>(is_k ? p.k_out : p.q_out);
  const int64_t x_token = is_k ? p.k_token : p.q_token, x_head = is_k ? p.k_head : p.q_head;
  const int64_t y_token = is_k ? p.dyk_token : p.dyq_token, y_head = is_k ? p.dyk_head : p.dyq_head;
  const int64_t d_token = is_k ? p.k_out_token : p.q_out_token;
  const int64_t d_head = is_k ? p.k_out_head : p.q_out_head;
  int oa[KU], ob[KU], have = 0;
#pragma unroll
  for (int k = 0; k < KU; ++k) {
    unit_at<VEC, HALF>(gl + k * ln, ru, half, oa[k], ob[k]);
    if (gl + k * ln < U) have = k + 1;
  }
  uint64_t da[N2], db[N2];  // the weight's gradient
#pragma unroll
  for (int i = 0; i < N2; ++i) da[i] = db[i] = 0;
  const float inv_d = 1.f / p.d;
  const float* const wt = sh.w + (is_k ? p.d : 0);
  fill_fixed<DT, VEC, HALF>(p, sh);
  const RowSteps steps(ln, rows, tok, static_cast<int64_t>(ctas) * tok);
  const int64_t begin = static_cast<int64_t>(blockIdx.x - (is_k ? ctas_q : 0)) * tok;
  RowWalk w, ahead;
  steps.start(ahead, p, begin);
  uint32_t in = 0, out = 0;  // rounds fetched and taken
  auto fetch = [&] {
    if (ahead.t0 < p.T) {
      if (ahead.tk < ahead.tokens(p, tok)) {
        const int64_t t = ahead.t0 + ahead.tk;
        const uint32_t at = smem_u32(ring) + in % kStages * (kRing / kStages);
        X::fetch(at, px + t * x_token + ahead.r * x_head, oa, ob, have);
        X::fetch(at + 2 * KU * (kRopeThreads * 16), py + t * y_token + ahead.r * y_head, oa, ob, have);
      }
      if (!steps.next(ahead)) steps.start(ahead, p, ahead.t0 + steps.step);
    }
    copy_commit();
    ++in;
  };
  if constexpr (VEC > 1) {
#pragma unroll 1
    for (int i = 0; i < kStages - 1; ++i) fetch();
  }
  for (int64_t t0 = begin; t0 < p.T; t0 += steps.step) {
    steps.start(w, p, t0);
    const int nt = w.tokens(p, tok);
    if (threadIdx.x < nt * p.axes) {
      const int a = threadIdx.x / nt, i = threadIdx.x - a * nt;
      s_pos[a][i] = p.pos[a * p.T + t0 + i];
    }
    __syncthreads();  // also: the last batch's sines have been read
    fill_angles<VEC>(p, nt, sh, true, [&](int a, int i) { return s_pos[a][i]; });
    __syncthreads();
    bool more = true;
    while (more) {
      const bool live = w.tk < nt;
      T* const dst = pd + (t0 + w.tk) * d_token + w.r * d_head;
      X x, dy;
      if constexpr (VEC > 1) {
        copy_wait<kStages - 2>();
        const uint8_t* const at = ring + out++ % kStages * (kRing / kStages);
        x.take(at, live ? have : 0);
        dy.take(at + 2 * KU * (kRopeThreads * 16), live ? have : 0);
        fetch();
      } else {
        x.clear();
        dy.clear();
        if (live) {
          x.load(px + (t0 + w.tk) * x_token + w.r * x_head, oa, ob, have);
          dy.load(py + (t0 + w.tk) * y_token + w.r * y_head, oa, ob, have);
        }
      }
      uint64_t A[N2], B[N2], gA[N2], gB[N2];
      x.widen(A, B);
      dy.widen(gA, gB);
      if (live) turn<VEC, N2>(gA, gB, sh.cs + w.tk * half, gl, ln, ru);
      more = steps.next(w);
      uint64_t ss2 = 0, sg2 = 0;
#pragma unroll
      for (int i = 0; i < N2; ++i) {
        uint64_t wa, wb;
        pairs_of<VEC>(wt, i, gl, ln, U, wa, wb);
        ss2 = f2_fma(A[i], A[i], f2_fma(B[i], B[i], ss2));
        sg2 = f2_fma(f2_mul(gA[i], A[i]), wa, f2_fma(f2_mul(gB[i], B[i]), wb, sg2));
      }
      const float ss = sum_lanes(f2_sum(ss2), ln), sg = sum_lanes(f2_sum(sg2), ln);
      if (!live) continue;
      const float rr = rsqrtf(fmaf(ss, inv_d, p.eps)), c = -rr * rr * rr * (sg * inv_d);
      const uint64_t rr2 = f2(rr, rr), c2 = f2(c, c);
#pragma unroll
      for (int i = 0; i < N2; ++i) {
        uint64_t wa, wb;
        pairs_of<VEC>(wt, i, gl, ln, U, wa, wb);
        const uint64_t ga = f2_mul(gA[i], rr2), gb = f2_mul(gB[i], rr2);
        da[i] = f2_fma(ga, A[i], da[i]);
        db[i] = f2_fma(gb, B[i], db[i]);
        A[i] = f2_fma(A[i], c2, f2_mul(ga, wa));
        B[i] = f2_fma(B[i], c2, f2_mul(gb, wb));
      }
      X::store(dst, oa, ob, have, A, B);
    }
  }
  if (!p.part) return;
  // the groups of a warp, then the warps
  __shared__ float s_dw[kRopeThreads / 32][512];
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
#pragma unroll
  for (int i = 0; i < N2; ++i) {
    float v[4];  // A, A of the next pair, B, B
    f2_split(da[i], v[0], v[1]);
    f2_split(db[i], v[2], v[3]);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      for (int o = ln; o < 32; o *= 2) v[j] += __shfl_xor_sync(kAll, v[j], o);
      const int n = 2 * i + j % 2, k = n / VEC, e = n % VEC;
      const int at = HALF || VEC == 1 ? (j < 2 ? oa[k] : ob[k]) + e : oa[k] + 2 * e + j / 2;
      if (lane < ln && k < have) s_dw[warp][at] = v[j];
    }
  }
  __syncthreads();
  for (int i = threadIdx.x; i < p.d; i += kRopeThreads) {
    float s = 0.f;
#pragma unroll
    for (int x = 0; x < kRopeThreads / 32; ++x) s += s_dw[x][i];
    p.part[static_cast<size_t>(blockIdx.x) * p.d + i] = s;
  }
}

// Column c of the CTAs' partial sums [ctas][d], the first ctas_q rows of q's weight, the others of
// k's: 32 columns and 32 shares of the rows per CTA; blockIdx.y picks the weight.
__global__ void __launch_bounds__(1024)
    norm_rope_sum_kernel(const float* part, int ctas, int ctas_q, int d, float* dq_weight,
                         float* dk_weight) {
  __shared__ float s[32][33];
  float* const out = blockIdx.y ? dk_weight : dq_weight;
  if (!out) return;
  const int lane = threadIdx.x % 32, share = threadIdx.x / 32, c = blockIdx.x * 32 + lane;
  const int from = blockIdx.y ? ctas_q : 0, to = blockIdx.y ? ctas : ctas_q;
  float x = 0.f;
  if (c < d)
    for (int i = from + share; i < to; i += 32) x += part[static_cast<size_t>(i) * d + c];
  s[share][lane] = x;
  __syncthreads();
  x = s[lane][share];  // lane: share; share: column
#pragma unroll
  for (int o = 16; o > 0; o /= 2) x += __shfl_xor_sync(kAll, x, o);
  const int col = blockIdx.x * 32 + share;
  if (lane == 0 && col < d) out[col] = x;
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

// Tokens of a batch: the least time, in rounds of a CTA's groups of lanes over rows. A CTA has a whole
// number of batches, and a batch takes as many rounds as its rows need and about two for its angles
// and barriers.
constexpr int kMostShared = 81920;  // of the forward; the gradient's is at most twice that
struct Share {  // rows of a token, and the CTAs that share the tokens
  int rows, ctas;
};
int tokens_of(const NormRopeParams& p, int ln, Share a, Share b) {
  const int groups = kRopeThreads / ln;
  int best = 1;
  int64_t least = INT64_MAX;
  for (int tok = 1; tok <= kTokMax; ++tok) {
    if (tok > 1 && shared_bytes(tok, p.rot / 2, p.d) > 16384) break;
    const int64_t batches = (p.T + tok - 1) / tok;
    int64_t cost = 0;
    for (const Share& s : {a, b})
      if (s.rows)
        cost = std::max(cost, (batches + s.ctas - 1) / s.ctas *
                                  ((static_cast<int64_t>(s.rows) * tok + groups - 1) / groups + 2));
    if (cost < least) {
      least = cost;
      best = tok;
    }
  }
  return best;
}

template <int DT, int VEC, int KU, int MODE>
cudaError_t launch_v(const NormRopeParams& p, bool half_style, int sms, cudaStream_t stream) {
  const int ln = lanes_of(p.d / (2 * VEC), KU), rows = p.H + (MODE ? 2 : 1) * p.Hkv;
  const int tok = tokens_of(p, ln, Share{rows, 4 * sms}, Share{0, 1});
  const int smem = static_cast<int>(shared_bytes(tok, p.rot / 2, p.d)) + ring_bytes<VEC>(2 * KU);
  const int64_t grid = std::min<int64_t>((p.T + tok - 1) / tok, 4 * sms);
  auto* k = half_style ? norm_rope_kernel<DT, VEC, KU, true, MODE>
                       : norm_rope_kernel<DT, VEC, KU, false, MODE>;
  const cudaError_t e = half_style ? prepare_kernel<norm_rope_kernel<DT, VEC, KU, true, MODE>>(kMostShared)
                                   : prepare_kernel<norm_rope_kernel<DT, VEC, KU, false, MODE>>(kMostShared);
  if (e != cudaSuccess) return e;
  k<<<static_cast<unsigned>(grid), kRopeThreads, smem, stream>>>(p, tok, ln);
  return cudaGetLastError();
}
template <int DT, int VEC, int KU>
cudaError_t launch_bwd_v(const NormRopeParams& p, bool half_style, int sms, cudaStream_t stream) {
  const int ln = lanes_of(p.d / (2 * VEC), KU);
  // CTAs of q and k by their heads, at least one each
  const int most = std::min(2 * sms, kNormCtas);
  int ctas_k = p.Hkv ? std::max<int>(1, static_cast<int64_t>(most) * p.Hkv / (p.H + p.Hkv)) : 0;
  int ctas_q = most - ctas_k;
  const int tok = tokens_of(p, ln, Share{p.H, ctas_q}, Share{p.Hkv, ctas_k});
  const int smem = static_cast<int>(shared_bytes(tok, p.rot / 2, p.d)) + ring_bytes<VEC>(4 * KU);
  const int64_t batches = (p.T + tok - 1) / tok;
  ctas_q = static_cast<int>(std::min<int64_t>(ctas_q, batches));
  ctas_k = static_cast<int>(std::min<int64_t>(ctas_k, batches));
  auto* k = half_style ? norm_rope_bwd_kernel<DT, VEC, KU, true>
                       : norm_rope_bwd_kernel<DT, VEC, KU, false>;
  cudaError_t e = half_style ? prepare_kernel<norm_rope_bwd_kernel<DT, VEC, KU, true>>(2 * kMostShared)
                             : prepare_kernel<norm_rope_bwd_kernel<DT, VEC, KU, false>>(2 * kMostShared);
  if (e != cudaSuccess) return e;
  k<<<ctas_q + ctas_k, kRopeThreads, smem, stream>>>(p, tok, ln, ctas_q);
  e = cudaGetLastError();
  if (e != cudaSuccess || !p.part) return e;
  norm_rope_sum_kernel<<<dim3((p.d + 31) / 32, 2), 1024, 0, stream>>>(
      p.part, ctas_q + ctas_k, ctas_q, p.d, p.dq_weight, p.dk_weight);
  return cudaGetLastError();
}

template <int DT, int MODE>
cudaError_t launch_m(const NormRopeParams& p, bool half_style, bool vec, int sms,
                     cudaStream_t stream) {
  if (!vec) return launch_v<DT, 1, 8, MODE>(p, half_style, sms, stream);
  if constexpr (DT == FA_F32)
    return launch_v<DT, 4, 2, MODE>(p, half_style, sms, stream);
  else
    return launch_v<DT, 8, 1, MODE>(p, half_style, sms, stream);
}
template <int DT>
cudaError_t launch_bwd_t(const NormRopeParams& p, bool half_style, bool vec, int sms,
                         cudaStream_t stream) {
  if (!vec) return launch_bwd_v<DT, 1, 8>(p, half_style, sms, stream);
  if constexpr (DT == FA_F32)
    return launch_bwd_v<DT, 4, 2>(p, half_style, sms, stream);
  else
    return launch_bwd_v<DT, 8, 1>(p, half_style, sms, stream);
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
