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

// A CTA's shared memory: sines and cosines of its tokens, the frequencies, the weights of q and k,
// the pairs' axes. Neighbouring units lie next to each other, 16 bytes of a unit at a time where it
// has that many, so that neighbouring lanes read neighbouring 16 bytes.
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

__device__ __forceinline__ float weight_at(const void* w, int f32, int dt, int i) {
  if (!w) return 1.f;
  if (f32) return static_cast<const float*>(w)[i];
  const uint16_t x = static_cast<const uint16_t*>(w)[i];
  return dt == FA_BF16 ? Elem<FA_BF16>::get(x) : Elem<FA_F16>::get(x);
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
  constexpr int W = VEC == 1 ? 2 : 4;  // floats of a unit next to each other
  for (int i = threadIdx.x; i < 2 * p.d; i += kRopeThreads) {
    const int kind = i / p.d, j = i - kind * p.d, u = j / (2 * VEC), e = j % (2 * VEC);
    int oa, ob;
    unit_at<VEC, HALF>(u, ru, half, oa, ob);
    const int c = e < VEC ? oa + e : ob + e - VEC;
    sh.w[kind * p.d + ((e / W) * U + u) * W + e % W] =
        weight_at(kind ? p.k_weight : p.q_weight, p.w_f32, DT, c);
  }
}
// Sines and cosines of nt tokens; pos(axis, token) in 64 bits.
template <int VEC, typename Pos>
__device__ __forceinline__ void fill_angles(const NormRopeParams& p, int nt, const Shared& sh,
                                            bool inverse, Pos pos) {
  const int half = p.rot / 2, ru = half / VEC;
  constexpr int W = VEC == 1 ? 1 : 2;  // pairs of a unit next to each other
  for (int i = threadIdx.x; i < nt * half; i += kRopeThreads) {
    const int tk = i / half, f = i - tk * half, u = f / VEC, e = f % VEC;
    const int64_t at = pos(sh.axis[f], tk);
    const uint64_t phase = static_cast<uint64_t>(inverse ? -at : at) * sh.freq[f];
    float s, c;  // the phase as a signed fraction of a turn: half turns in [-1, 1]
    sincospif(static_cast<float>(static_cast<int64_t>(phase)) * 1.08420217248550443e-19f, &s, &c);
    sh.cs[tk * half + ((e / W) * ru + u) * W + e % W] =
        make_float2(c * p.amplitude, s * p.amplitude);
  }
}

// The rotation of one unit's pairs.
template <int VEC, bool HALF>
__device__ __forceinline__ void turn(float* v, const float2* cs, int ru, int u) {
  auto pair = [&](int e, float c, float s) {
    constexpr bool kSplit = HALF || VEC == 1;  // pair e: e of both chunks, or 2e and 2e + 1
    float& xa = v[kSplit ? e : 2 * e];
    float& xb = v[kSplit ? VEC + e : 2 * e + 1];
    const float a = xa, b = xb;
    xa = a * c - b * s;
    xb = b * c + a * s;
  };
  if constexpr (VEC == 1) {
    pair(0, cs[u].x, cs[u].y);
  } else {
#pragma unroll
    for (int e = 0; e < VEC; e += 2) {
      const float4 k = *reinterpret_cast<const float4*>(cs + ((e / 2) * ru + u) * 2);
      pair(e, k.x, k.y);
      pair(e + 1, k.z, k.w);
    }
  }
}
// The weights of one unit.
template <int VEC>
__device__ __forceinline__ void unit_weights(const float* w, int U, int u, float* out) {
  if constexpr (VEC == 1) {
    out[0] = w[2 * u];
    out[1] = w[2 * u + 1];
  } else {
#pragma unroll
    for (int e = 0; e < 2 * VEC; e += 4) {
      const float4 k = *reinterpret_cast<const float4*>(w + ((e / 4) * U + u) * 4);
      out[e] = k.x, out[e + 1] = k.y, out[e + 2] = k.z, out[e + 3] = k.w;
    }
  }
}

// A lane's part of a row: KU units of VEC + VEC elements.
template <int DT, int VEC, int KU>
struct Part {
  using T = typename Elem<DT>::T;
  using C = Chunk<T, VEC>;
  C a[KU], b[KU];
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int k = 0; k < KU; ++k)
#pragma unroll
      for (int e = 0; e < VEC; ++e) a[k].e[e] = b[k].e[e] = T(0);
  }
  __device__ __forceinline__ void load(const void* row, const int* oa, const int* ob, int have) {
    const T* src = static_cast<const T*>(row);
#pragma unroll
    for (int k = 0; k < KU; ++k)
      if (k < have) {
        a[k] = *reinterpret_cast<const C*>(src + oa[k]);
        b[k] = *reinterpret_cast<const C*>(src + ob[k]);
      }
  }
  // elements 0 .. VEC-1 of unit k at v[k][0 ..], its others behind them
  __device__ __forceinline__ void widen(float (*v)[2 * VEC]) const {
#pragma unroll
    for (int k = 0; k < KU; ++k)
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        v[k][e] = Elem<DT>::get(a[k].e[e]);
        v[k][VEC + e] = Elem<DT>::get(b[k].e[e]);
      }
  }
  static __device__ __forceinline__ void store(void* row, const int* oa, const int* ob, int have,
                                               const float (*v)[2 * VEC]) {
    T* dst = static_cast<T*>(row);
#pragma unroll
    for (int k = 0; k < KU; ++k) {
      if (k >= have) continue;
      C a, b;
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        a.e[e] = Elem<DT>::put(v[k][e]);
        b.e[e] = Elem<DT>::put(v[k][VEC + e]);
      }
      *reinterpret_cast<C*>(dst + oa[k]) = a;
      *reinterpret_cast<C*>(dst + ob[k]) = b;
    }
  }
};
__device__ __forceinline__ float sum_lanes(float x, int ln) {
  for (int o = ln / 2; o > 0; o /= 2) x += __shfl_xor_sync(kAll, x, o);
  return x;
}

// The walk of a group of lanes over the rows of the CTA's tokens, (token, head) with the heads
// first: rows g, g + groups, ...
struct RowWalk {
  int tk, r, dt, dr, rows;
  __device__ __forceinline__ RowWalk(int g, int groups, int rows)
      : tk(g / rows), r(g % rows), dt(groups / rows), dr(groups % rows), rows(rows) {}
  __device__ __forceinline__ void next() {
    tk += dt;
    r += dr;
    if (r >= rows) {
      r -= rows;
      ++tk;
    }
  }
};

// Rows r of a token: H of q, Hkv of k and, when appending, Hkv of v. MODE 0: y to q_out and k_out;
// 1 and 2: q to q_out, k and v to the cache's slot of the token, in 16 and in 8 bits.
template <int DT, int VEC, int KU, bool HALF, int MODE>
__global__ void __launch_bounds__(kRopeThreads)
    norm_rope_kernel(const __grid_constant__ NormRopeParams p, int tok, int ln) {
  using T = typename Elem<DT>::T;
  extern __shared__ float4 s_dyn[];
  __shared__ int64_t s_dst[kTokMax], s_pos[FA_MAX_AXES][kTokMax];
  __shared__ int s_seq[kTokMax];
  const int half = p.rot / 2, ru = half / VEC, U = p.d / (2 * VEC);
  const Shared sh(s_dyn, tok, half, p.d);
  const int64_t t0 = static_cast<int64_t>(blockIdx.x) * tok;
  const int nt = static_cast<int>(min(static_cast<int64_t>(tok), p.T - t0));
  const int groups = kRopeThreads / ln, gl = threadIdx.x % ln;
  const int rows = MODE ? p.H + 2 * p.Hkv : p.H + p.Hkv;
  int oa[KU], ob[KU], have = 0;
#pragma unroll
  for (int k = 0; k < KU; ++k) {
    unit_at<VEC, HALF>(gl + k * ln, ru, half, oa[k], ob[k]);
    if (gl + k * ln < U) have = k + 1;
  }
  RowWalk w(threadIdx.x / ln, groups, rows);
  auto row_at = [&]() -> const void* {
    const int64_t t = t0 + w.tk;
    if (w.r < p.H) return static_cast<const T*>(p.q) + t * p.q_token + w.r * p.q_head;
    if (w.r < p.H + p.Hkv)
      return static_cast<const T*>(p.k) + t * p.k_token + (w.r - p.H) * p.k_head;
    return static_cast<const T*>(p.v) + t * p.v_token +
           static_cast<int64_t>(w.r - p.H - p.Hkv) * p.d;
  };
  Part<DT, VEC, KU> x;
  x.clear();
  if (w.tk < nt) x.load(row_at(), oa, ob, have);  // under way while the angles are made
  fill_fixed<DT, VEC, HALF>(p, sh);
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
  __syncthreads();
  fill_angles<VEC>(p, nt, sh, p.inverse != 0, [&](int a, int i) { return s_pos[a][i]; });
  __syncthreads();

  const float inv_d = 1.f / p.d;
  for (int left = nt * rows; left > 0; left -= groups) {  // every lane goes round alike
    const bool live = w.tk < nt, is_v = MODE && w.r >= p.H + p.Hkv;
    const int r = w.r;
    const int64_t t = t0 + w.tk;
    float v[KU][2 * VEC];
    x.widen(v);
    if (p.norm) {
      float ss = 0.f;
#pragma unroll
      for (int k = 0; k < KU; ++k)
#pragma unroll
        for (int e = 0; e < 2 * VEC; ++e) ss = k < have ? fmaf(v[k][e], v[k][e], ss) : ss;
      ss = sum_lanes(ss, ln);
      if (!is_v) {
        const float rr = rsqrtf(fmaf(ss, inv_d, p.eps));
#pragma unroll
        for (int k = 0; k < KU; ++k) {
          if (k >= have) continue;
          float wt[2 * VEC];
          unit_weights<VEC>(sh.w + (r < p.H ? 0 : p.d), U, gl + k * ln, wt);
#pragma unroll
          for (int e = 0; e < 2 * VEC; ++e) v[k][e] *= rr * wt[e];
        }
      }
    }
    if (!is_v && live) {
#pragma unroll
      for (int k = 0; k < KU; ++k)
        if (gl + k * ln < ru) turn<VEC, HALF>(v[k], sh.cs + w.tk * half, ru, gl + k * ln);
    }
    const int64_t slot = MODE && live ? s_dst[w.tk] : 0;
    if (MODE == 2) {  // every group of the warp takes part in the shuffles
      uint32_t big = 0;
#pragma unroll
      for (int k = 0; k < KU; ++k)
#pragma unroll
        for (int e = 0; e < 2 * VEC; ++e)
          if (k < have) big = max(big, __float_as_uint(v[k][e]) & 0x7fffffffu);
      for (int o = ln / 2; o > 0; o /= 2) big = max(big, __shfl_xor_sync(kAll, big, o));
      if (live && r >= p.H && slot >= 0) {
        const int h = r - p.H - (is_v ? p.Hkv : 0), byte = power_byte(big);
        const float up = byte == 255 ? 0.f : up_of(byte);
        const int64_t row = slot + static_cast<int64_t>(h) * p.page_size;
        uint8_t* dst = static_cast<uint8_t*>(is_v ? p.v_pages : p.k_pages) + row * p.d;
        if (gl == 0) (is_v ? p.v_scales : p.k_scales)[row] = static_cast<uint8_t>(byte);
#pragma unroll
        for (int k = 0; k < KU; ++k) {
          if (k >= have) continue;
          Chunk<uint8_t, VEC> a, b;
#pragma unroll
          for (int e = 0; e < VEC; e += 2) {
            const int e1 = e + 1 < VEC ? e + 1 : e;
            uint32_t lo = cvt_e4m3x2(v[k][e] * up, v[k][e1] * up);
            uint32_t hi = cvt_e4m3x2(v[k][VEC + e] * up, v[k][VEC + e1] * up);
            if (byte == 255) lo = hi = 0;
            a.e[e] = static_cast<uint8_t>(lo);
            b.e[e] = static_cast<uint8_t>(hi);
            if (VEC > 1) {
              a.e[e1] = static_cast<uint8_t>(lo >> 8);
              b.e[e1] = static_cast<uint8_t>(hi >> 8);
            }
          }
          *reinterpret_cast<Chunk<uint8_t, VEC>*>(dst + oa[k]) = a;
          *reinterpret_cast<Chunk<uint8_t, VEC>*>(dst + ob[k]) = b;
        }
      }
    }
    w.next();
    if (w.tk < nt) x.load(row_at(), oa, ob, have);  // of the row to come
    if (!live || (MODE && (r < p.H ? slot == -2 : MODE == 2 || slot < 0))) continue;
    T* dst;
    if (r < p.H)
      dst = static_cast<T*>(p.q_out) + t * p.q_out_token + r * p.q_out_head;
    else if (MODE == 0)
      dst = static_cast<T*>(p.k_out) + t * p.k_out_token + (r - p.H) * p.k_out_head;
    else
      dst = static_cast<T*>(is_v ? p.v_pages : p.k_pages) +
            (slot + static_cast<int64_t>(r - p.H - (is_v ? p.Hkv : 0)) * p.page_size) * p.d;
    Part<DT, VEC, KU>::store(dst, oa, ob, have, v);
  }
}

// The gradient. Persistent, CTAs 0 .. ctas_q - 1 for the heads of q, the others for those of k, each
// over every ctas'th batch of tokens. A thread has the same elements of every row, so the weight's
// gradient adds up in its registers; they meet once at the end, per CTA, in a fixed order, and
// norm_rope_sum_kernel adds the CTAs in theirs: the same bits on every run of the same sizes.
template <int DT, int VEC, int KU, bool HALF>
__global__ void __launch_bounds__(kRopeThreads, VEC == 8 ? 2 : 1)
    norm_rope_bwd_kernel(const __grid_constant__ NormRopeParams p, int tok, int ln, int ctas_q) {
  using T = typename Elem<DT>::T;
  extern __shared__ float4 s_dyn[];
  __shared__ int64_t s_pos[FA_MAX_AXES][kTokMax];
  const int half = p.rot / 2, ru = half / VEC, U = p.d / (2 * VEC);
  const Shared sh(s_dyn, tok, half, p.d);
  const int groups = kRopeThreads / ln, gl = threadIdx.x % ln;
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
  float dw[KU][2 * VEC];
#pragma unroll
  for (int k = 0; k < KU; ++k)
#pragma unroll
    for (int e = 0; e < 2 * VEC; ++e) dw[k][e] = 0.f;
  const float inv_d = 1.f / p.d;
  const float* const wt = sh.w + (is_k ? p.d : 0);
  fill_fixed<DT, VEC, HALF>(p, sh);
  for (int64_t t0 = static_cast<int64_t>(blockIdx.x - (is_k ? ctas_q : 0)) * tok; t0 < p.T;
       t0 += static_cast<int64_t>(ctas) * tok) {
    const int nt = static_cast<int>(min(static_cast<int64_t>(tok), p.T - t0));
    RowWalk w(threadIdx.x / ln, groups, rows);
    Part<DT, VEC, KU> x, dy;
    x.clear();
    dy.clear();
    auto load = [&] {
      const int64_t t = t0 + w.tk;
      x.load(px + t * x_token + w.r * x_head, oa, ob, have);
      dy.load(py + t * y_token + w.r * y_head, oa, ob, have);
    };
    if (w.tk < nt) load();
    if (threadIdx.x < nt * p.axes) {
      const int a = threadIdx.x / nt, i = threadIdx.x - a * nt;
      s_pos[a][i] = p.pos[a * p.T + t0 + i];
    }
    __syncthreads();  // also: the last batch's sines have been read
    fill_angles<VEC>(p, nt, sh, true, [&](int a, int i) { return s_pos[a][i]; });
    __syncthreads();
    for (int left = nt * rows; left > 0; left -= groups) {
      const bool live = w.tk < nt;
      T* const dst = pd + (t0 + w.tk) * d_token + w.r * d_head;
      float v[KU][2 * VEC], g[KU][2 * VEC];
      x.widen(v);
      dy.widen(g);
      float ss = 0.f, sg = 0.f;
      if (live) {
#pragma unroll
        for (int k = 0; k < KU; ++k)
          if (gl + k * ln < ru) turn<VEC, HALF>(g[k], sh.cs + w.tk * half, ru, gl + k * ln);
      }
      w.next();
      if (w.tk < nt) load();  // of the row to come
#pragma unroll
      for (int k = 0; k < KU; ++k) {
        if (k >= have) continue;
        float wk[2 * VEC];
        unit_weights<VEC>(wt, U, gl + k * ln, wk);
#pragma unroll
        for (int e = 0; e < 2 * VEC; ++e) {
          ss = fmaf(v[k][e], v[k][e], ss);
          sg = fmaf(wk[e] * g[k][e], v[k][e], sg);
        }
      }
      ss = sum_lanes(ss, ln);
      sg = sum_lanes(sg, ln);
      if (!live) continue;
      const float rr = rsqrtf(fmaf(ss, inv_d, p.eps)), c = rr * rr * rr * (sg * inv_d);
#pragma unroll
      for (int k = 0; k < KU; ++k) {
        if (k >= have) continue;
        float wk[2 * VEC];
        unit_weights<VEC>(wt, U, gl + k * ln, wk);
#pragma unroll
        for (int e = 0; e < 2 * VEC; ++e) {
          dw[k][e] = fmaf(g[k][e] * v[k][e], rr, dw[k][e]);
          v[k][e] = fmaf(-v[k][e], c, rr * (wk[e] * g[k][e]));
        }
      }
      Part<DT, VEC, KU>::store(dst, oa, ob, have, v);
    }
  }
  if (!p.part) return;
  // the groups of a warp, then the warps
  __shared__ float s_dw[kRopeThreads / 32][512];
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
#pragma unroll
  for (int k = 0; k < KU; ++k)
#pragma unroll
    for (int e = 0; e < 2 * VEC; ++e) {
      float s = dw[k][e];
      for (int o = ln; o < 32; o *= 2) s += __shfl_xor_sync(kAll, s, o);
      if (lane < ln && k < have) s_dw[warp][(e < VEC ? oa[k] : ob[k] - VEC) + e] = s;
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

// Tokens of a CTA: as many as give every group of lanes `each` rows, where that leaves every SM a few
// CTAs and their sines fit (the angles' cost is shared by more heads than by more tokens).
int tokens_of(const NormRopeParams& p, int ln, int rows, int each, int64_t ctas) {
  const int groups = kRopeThreads / ln;
  int64_t tok = std::max(1, each * groups / rows);
  tok = std::min<int64_t>({tok, kTokMax, std::max<int64_t>(1, p.T / ctas)});
  while (tok > 1 && shared_bytes(static_cast<int>(tok), p.rot / 2, p.d) > 16384) --tok;
  return static_cast<int>(tok);
}

template <int DT, int VEC, int KU, int MODE>
cudaError_t launch_v(const NormRopeParams& p, bool half_style, int sms, cudaStream_t stream) {
  const int ln = lanes_of(p.d / (2 * VEC), KU), rows = p.H + (MODE ? 2 : 1) * p.Hkv;
  const int tok = tokens_of(p, ln, rows, 4, 8LL * sms);
  const size_t smem = shared_bytes(tok, p.rot / 2, p.d);
  const int64_t grid = (p.T + tok - 1) / tok;
  if (grid > 0x7fffffff) return cudaErrorInvalidConfiguration;
  auto* k = half_style ? norm_rope_kernel<DT, VEC, KU, true, MODE>
                       : norm_rope_kernel<DT, VEC, KU, false, MODE>;
  k<<<static_cast<unsigned>(grid), kRopeThreads, smem, stream>>>(p, tok, ln);
  return cudaGetLastError();
}
template <int DT, int VEC, int KU>
cudaError_t launch_bwd_v(const NormRopeParams& p, bool half_style, int sms, cudaStream_t stream) {
  const int ln = lanes_of(p.d / (2 * VEC), KU);
  const int tok = tokens_of(p, ln, std::max(1, std::min(p.H, p.Hkv ? p.Hkv : p.H)), 4, 4LL * sms);
  const size_t smem = shared_bytes(tok, p.rot / 2, p.d);
  const int64_t batches = (p.T + tok - 1) / tok;
  const int64_t most = std::min<int64_t>(2 * sms, kNormCtas);
  // CTAs of q and k by their heads, at least one each
  const int all = static_cast<int>(std::min<int64_t>(most, p.Hkv ? 2 * batches : batches));
  int ctas_k = p.Hkv ? static_cast<int>(static_cast<int64_t>(all) * p.Hkv / (p.H + p.Hkv)) : 0;
  if (p.Hkv) ctas_k = std::max(1, ctas_k);
  int ctas_q = std::max(1, all - ctas_k);
  ctas_q = static_cast<int>(std::min<int64_t>(ctas_q, batches));
  ctas_k = static_cast<int>(std::min<int64_t>(ctas_k, batches));
  auto* k = half_style ? norm_rope_bwd_kernel<DT, VEC, KU, true>
                       : norm_rope_bwd_kernel<DT, VEC, KU, false>;
  k<<<ctas_q + ctas_k, kRopeThreads, smem, stream>>>(p, tok, ln, ctas_q);
  cudaError_t e = cudaGetLastError();
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
