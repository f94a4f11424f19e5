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
#include <cstdint>

#include "fa_ptx.cuh"
#include "fa_rope.cuh"

namespace fa {
namespace {

constexpr int kTokMax = 4;  // tokens of a CTA
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

// Sines and cosines of the CTA's tokens, [token][e][unit] for pair unit * VEC + e, so that
// neighbouring lanes read neighbouring words. pos(axis, token) in 64 bits.
template <int VEC, typename Pos>
__device__ __forceinline__ void fill_angles(const NormRopeParams& p, int nt, uint64_t* s_freq,
                                            uint8_t* s_axis, float2* s_cs, bool inverse, Pos pos) {
  const int half = p.rot / 2, ru = half / VEC;
  for (int i = threadIdx.x; i < nt * half; i += kRopeThreads) {
    const int tk = i / half, f = i - tk * half;
    const int64_t at = pos(s_axis[f], tk);
    const uint64_t phase = static_cast<uint64_t>(inverse ? -at : at) * s_freq[f];
    float s, c;  // the phase as a signed fraction of a turn: half turns in [-1, 1]
    sincospif(static_cast<float>(static_cast<int64_t>(phase)) * 1.08420217248550443e-19f, &s, &c);
    s_cs[tk * half + (f % VEC) * ru + f / VEC] = make_float2(c * p.amplitude, s * p.amplitude);
  }
}
__device__ __forceinline__ void fill_freqs(const NormRopeParams& p, uint64_t* s_freq,
                                           uint8_t* s_axis) {
  for (int i = threadIdx.x; i < p.rot / 2; i += kRopeThreads) {
    s_freq[i] = turns_q64(p.freqs[i]);
    int a = p.pair_axis ? p.pair_axis[i] : 0;
    if (a < 0 || a >= p.axes) {
      if (blockIdx.x == 0) atomicOr(p.status, FA_DEV_BAD_PAGE);
      a = 0;
    }
    s_axis[i] = static_cast<uint8_t>(a);
  }
}

// A lane's part of a row: KU units of VEC + VEC elements.
template <int DT, int VEC, int KU>
struct Part {
  using T = typename Elem<DT>::T;
  using C = Chunk<T, VEC>;
  C a[KU], b[KU];
};
// x of the lane's units; elements 0 .. VEC-1 of unit k at v[k][0 ..], its others behind them.
template <int DT, int VEC, int KU>
__device__ __forceinline__ void widen(const Part<DT, VEC, KU>& x, float (*v)[2 * VEC]) {
#pragma unroll
  for (int k = 0; k < KU; ++k)
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      v[k][e] = Elem<DT>::get(x.a[k].e[e]);
      v[k][VEC + e] = Elem<DT>::get(x.b[k].e[e]);
    }
}
// The rotation of one unit's pairs by (cos, sin) of cs.
template <int VEC, bool HALF>
__device__ __forceinline__ void turn(float* v, const float2* cs) {
#pragma unroll
  for (int e = 0; e < VEC; ++e) {
    constexpr bool kSplit = HALF || VEC == 1;  // pair e: e of both chunks, or 2e and 2e + 1
    float& xa = v[kSplit ? e : 2 * e];
    float& xb = v[kSplit ? VEC + e : 2 * e + 1];
    const float a = xa, b = xb;
    xa = a * cs[e].x - b * cs[e].y;
    xb = b * cs[e].x + a * cs[e].y;
  }
}
__device__ __forceinline__ float sum_lanes(float x, int ln) {
  for (int o = ln / 2; o > 0; o /= 2) x += __shfl_xor_sync(kAll, x, o);
  return x;
}
__device__ __forceinline__ float weight_at(const void* w, int f32, int dt, int i) {
  if (!w) return 1.f;
  if (f32) return static_cast<const float*>(w)[i];
  const uint16_t x = static_cast<const uint16_t*>(w)[i];
  return dt == FA_BF16 ? Elem<FA_BF16>::get(x) : Elem<FA_F16>::get(x);
}
template <int DT, int VEC, int KU>
__device__ __forceinline__ void load_weight(const void* w, int f32, const int* oa, const int* ob,
                                            int have, float (*v)[2 * VEC]) {
#pragma unroll
  for (int k = 0; k < KU; ++k)
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      v[k][e] = k < have ? weight_at(w, f32, DT, oa[k] + e) : 0.f;
      v[k][VEC + e] = k < have ? weight_at(w, f32, DT, ob[k] + e) : 0.f;
    }
}

// Rows r of a token: H of q, Hkv of k and, when appending, Hkv of v. MODE 0: y to q_out and k_out;
// 1 and 2: q to q_out, k and v to the cache's slot of the token, in 16 and in 8 bits.
template <int DT, int VEC, int KU, bool HALF, int MODE>
__global__ void __launch_bounds__(kRopeThreads)
    norm_rope_kernel(const __grid_constant__ NormRopeParams p, int tok, int ln) {
  using T = typename Elem<DT>::T;
  using C = Chunk<T, VEC>;
  extern __shared__ float2 s_cs[];
  __shared__ int64_t s_dst[kTokMax], s_pos[4][kTokMax];
  __shared__ int s_seq[kTokMax];
  const int half = p.rot / 2, ru = half / VEC, U = p.d / (2 * VEC);
  uint64_t* s_freq = reinterpret_cast<uint64_t*>(s_cs + static_cast<size_t>(tok) * half);
  uint8_t* s_axis = reinterpret_cast<uint8_t*>(s_freq + half);
  const int64_t t0 = static_cast<int64_t>(blockIdx.x) * tok;
  const int nt = static_cast<int>(min(static_cast<int64_t>(tok), p.T - t0));
  const int groups = kRopeThreads / ln, step = groups / tok;
  const int g = threadIdx.x / ln, gl = threadIdx.x % ln, tk = g / step;
  const int rows = MODE ? p.H + 2 * p.Hkv : p.H + p.Hkv;
  const int64_t t = t0 + tk;
  int oa[KU], ob[KU], have = 0;
#pragma unroll
  for (int k = 0; k < KU; ++k) {
    unit_at<VEC, HALF>(gl + k * ln, ru, half, oa[k], ob[k]);
    if (gl + k * ln < U) have = k + 1;
  }
  auto load = [&](int r, Part<DT, VEC, KU>& x) {
    const T* src;
    if (r < p.H)
      src = static_cast<const T*>(p.q) + t * p.q_token + r * p.q_head;
    else if (r < p.H + p.Hkv)
      src = static_cast<const T*>(p.k) + t * p.k_token + (r - p.H) * p.k_head;
    else
      src = static_cast<const T*>(p.v) + t * p.v_token +
            static_cast<int64_t>(r - p.H - p.Hkv) * p.d;
#pragma unroll
    for (int k = 0; k < KU; ++k)
      if (k < have) {
        x.a[k] = *reinterpret_cast<const C*>(src + oa[k]);
        x.b[k] = *reinterpret_cast<const C*>(src + ob[k]);
      }
  };
  Part<DT, VEC, KU> cur, next;
#pragma unroll
  for (int k = 0; k < KU; ++k)
#pragma unroll
    for (int e = 0; e < VEC; ++e)
      cur.a[k].e[e] = cur.b[k].e[e] = next.a[k].e[e] = next.b[k].e[e] = T(0);
  int r = g % step;
  if (tk < nt && r < rows) load(r, cur);  // under way while the angles are made
  fill_freqs(p, s_freq, s_axis);
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
  fill_angles<VEC>(p, nt, s_freq, s_axis, s_cs, p.inverse != 0,
                   [&](int a, int i) { return s_pos[a][i]; });
  __syncthreads();

  float2 cs[KU][VEC];
#pragma unroll
  for (int k = 0; k < KU; ++k)
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      const int u = gl + k * ln;
      cs[k][e] = tk < nt && u < ru ? s_cs[tk * half + e * ru + u] : make_float2(1.f, 0.f);
    }
  float w[KU][2 * VEC];
  int kind = -1;  // whose weight w holds
  const float inv_d = 1.f / p.d;
  const int64_t slot = MODE && tk < nt ? s_dst[tk] : 0;
  for (int r1 = 0; r1 < rows; r1 += step, r += step) {  // every lane of a warp goes round alike
    const bool live = tk < nt && r < rows;
    if (tk < nt && r + step < rows) load(r + step, next);
    float v[KU][2 * VEC];
    widen<DT, VEC, KU>(cur, v);
    cur = next;
    const bool is_v = r >= p.H + p.Hkv;
    if (p.norm) {
      float ss = 0.f;
#pragma unroll
      for (int k = 0; k < KU; ++k)
#pragma unroll
        for (int e = 0; e < 2 * VEC; ++e) ss = k < have ? fmaf(v[k][e], v[k][e], ss) : ss;
      ss = sum_lanes(ss, ln);
      if (!is_v) {
        if (kind != (r >= p.H)) {
          kind = r >= p.H;
          load_weight<DT, VEC, KU>(kind ? p.k_weight : p.q_weight, p.w_f32, oa, ob, have, w);
        }
        const float rr = rsqrtf(fmaf(ss, inv_d, p.eps));
#pragma unroll
        for (int k = 0; k < KU; ++k)
#pragma unroll
          for (int e = 0; e < 2 * VEC; ++e) v[k][e] *= rr * w[k][e];
      }
    }
    if (!is_v) {
#pragma unroll
      for (int k = 0; k < KU; ++k)
        if (gl + k * ln < ru) turn<VEC, HALF>(v[k], cs[k]);
    }
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
            uint32_t x = cvt_e4m3x2(v[k][e] * up, v[k][e1] * up);
            uint32_t y = cvt_e4m3x2(v[k][VEC + e] * up, v[k][VEC + e1] * up);
            if (byte == 255) x = y = 0;
            a.e[e] = static_cast<uint8_t>(x);
            b.e[e] = static_cast<uint8_t>(y);
            if (VEC > 1) {
              a.e[e1] = static_cast<uint8_t>(x >> 8);
              b.e[e1] = static_cast<uint8_t>(y >> 8);
            }
          }
          *reinterpret_cast<Chunk<uint8_t, VEC>*>(dst + oa[k]) = a;
          *reinterpret_cast<Chunk<uint8_t, VEC>*>(dst + ob[k]) = b;
        }
      }
      if (r >= p.H) continue;
    }
    if (!live || (MODE && (r < p.H ? slot == -2 : slot < 0))) continue;
    T* dst;
    if (r < p.H)
      dst = static_cast<T*>(p.q_out) + t * p.q_out_token + r * p.q_out_head;
    else if (MODE == 0)
      dst = static_cast<T*>(p.k_out) + t * p.k_out_token + (r - p.H) * p.k_out_head;
    else
      dst = static_cast<T*>(is_v ? p.v_pages : p.k_pages) +
            (slot + static_cast<int64_t>(r - p.H - (is_v ? p.Hkv : 0)) * p.page_size) * p.d;
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
}

// The gradient. Persistent: CTA x takes the token batches x, x + gridDim.x, ..., a thread the same
// elements of every row, so the weights' gradients add up in its registers; they meet once at the
// end, per CTA, in a fixed order, and norm_rope_sum_kernel adds the CTAs in theirs: the same bits
// on every run of the same sizes.
template <int DT, int VEC, int KU, bool HALF>
__global__ void __launch_bounds__(kRopeThreads)
    norm_rope_bwd_kernel(const __grid_constant__ NormRopeParams p, int tok, int ln) {
  using T = typename Elem<DT>::T;
  using C = Chunk<T, VEC>;
  extern __shared__ float2 s_cs[];
  __shared__ int64_t s_pos[4][kTokMax];
  const int half = p.rot / 2, ru = half / VEC, U = p.d / (2 * VEC);
  uint64_t* s_freq = reinterpret_cast<uint64_t*>(s_cs + static_cast<size_t>(tok) * half);
  uint8_t* s_axis = reinterpret_cast<uint8_t*>(s_freq + half);
  const int groups = kRopeThreads / ln, step = groups / tok;
  const int g = threadIdx.x / ln, gl = threadIdx.x % ln, tk = g / step;
  const int rows = p.H + p.Hkv;
  int oa[KU], ob[KU], have = 0;
#pragma unroll
  for (int k = 0; k < KU; ++k) {
    unit_at<VEC, HALF>(gl + k * ln, ru, half, oa[k], ob[k]);
    if (gl + k * ln < U) have = k + 1;
  }
  float dw[2][KU][2 * VEC];
#pragma unroll
  for (int k = 0; k < KU; ++k)
#pragma unroll
    for (int e = 0; e < 2 * VEC; ++e) dw[0][k][e] = dw[1][k][e] = 0.f;
  const float inv_d = 1.f / p.d;
  fill_freqs(p, s_freq, s_axis);
  for (int64_t t0 = static_cast<int64_t>(blockIdx.x) * tok; t0 < p.T;
       t0 += static_cast<int64_t>(gridDim.x) * tok) {
    const int nt = static_cast<int>(min(static_cast<int64_t>(tok), p.T - t0));
    const int64_t t = t0 + tk;
    auto load = [&](int r, Part<DT, VEC, KU>& x, Part<DT, VEC, KU>& dy) {
      const T *src, *up;
      if (r < p.H) {
        src = static_cast<const T*>(p.q) + t * p.q_token + r * p.q_head;
        up = static_cast<const T*>(p.dyq) + t * p.dyq_token + r * p.dyq_head;
      } else {
        src = static_cast<const T*>(p.k) + t * p.k_token + (r - p.H) * p.k_head;
        up = static_cast<const T*>(p.dyk) + t * p.dyk_token + (r - p.H) * p.dyk_head;
      }
#pragma unroll
      for (int k = 0; k < KU; ++k)
        if (k < have) {
          x.a[k] = *reinterpret_cast<const C*>(src + oa[k]);
          x.b[k] = *reinterpret_cast<const C*>(src + ob[k]);
          dy.a[k] = *reinterpret_cast<const C*>(up + oa[k]);
          dy.b[k] = *reinterpret_cast<const C*>(up + ob[k]);
        }
    };
    Part<DT, VEC, KU> x, dy, nx, ndy;
#pragma unroll
    for (int k = 0; k < KU; ++k)
#pragma unroll
      for (int e = 0; e < VEC; ++e)
        x.a[k].e[e] = x.b[k].e[e] = dy.a[k].e[e] = dy.b[k].e[e] = nx.a[k].e[e] = nx.b[k].e[e] =
            ndy.a[k].e[e] = ndy.b[k].e[e] = T(0);
    int r = g % step;
    if (tk < nt && r < rows) load(r, x, dy);
    if (threadIdx.x < nt * p.axes) {
      const int a = threadIdx.x / nt, i = threadIdx.x - a * nt;
      s_pos[a][i] = p.pos[a * p.T + t0 + i];
    }
    __syncthreads();  // also: the last batch's sines have been read
    fill_angles<VEC>(p, nt, s_freq, s_axis, s_cs, true,
                     [&](int a, int i) { return s_pos[a][i]; });
    __syncthreads();
    float2 cs[KU][VEC];
#pragma unroll
    for (int k = 0; k < KU; ++k)
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        const int u = gl + k * ln;
        cs[k][e] = tk < nt && u < ru ? s_cs[tk * half + e * ru + u] : make_float2(1.f, 0.f);
      }
    float w[KU][2 * VEC];
    int kind = -1;
    for (int r1 = 0; r1 < rows; r1 += step, r += step) {
      const bool live = tk < nt && r < rows;
      if (tk < nt && r + step < rows) load(r + step, nx, ndy);
      float v[KU][2 * VEC], d[KU][2 * VEC];
      widen<DT, VEC, KU>(x, v);
      widen<DT, VEC, KU>(dy, d);
      x = nx;
      dy = ndy;
      if (kind != (r >= p.H)) {
        kind = r >= p.H;
        load_weight<DT, VEC, KU>(kind ? p.k_weight : p.q_weight, p.w_f32, oa, ob, have, w);
      }
#pragma unroll
      for (int k = 0; k < KU; ++k)
        if (gl + k * ln < ru) turn<VEC, HALF>(d[k], cs[k]);
      float ss = 0.f, sg = 0.f;
#pragma unroll
      for (int k = 0; k < KU; ++k)
#pragma unroll
        for (int e = 0; e < 2 * VEC; ++e)
          if (k < have) {
            ss = fmaf(v[k][e], v[k][e], ss);
            sg = fmaf(w[k][e] * d[k][e], v[k][e], sg);
          }
      ss = sum_lanes(ss, ln);
      sg = sum_lanes(sg, ln);
      if (!live) continue;
      const float rr = rsqrtf(fmaf(ss, inv_d, p.eps)), c = rr * rr * rr * (sg * inv_d);
      if (r < p.H) {
#pragma unroll
        for (int k = 0; k < KU; ++k)
#pragma unroll
          for (int e = 0; e < 2 * VEC; ++e) dw[0][k][e] = fmaf(d[k][e] * v[k][e], rr, dw[0][k][e]);
      } else {
#pragma unroll
        for (int k = 0; k < KU; ++k)
#pragma unroll
          for (int e = 0; e < 2 * VEC; ++e) dw[1][k][e] = fmaf(d[k][e] * v[k][e], rr, dw[1][k][e]);
      }
      T* dst = r < p.H ? static_cast<T*>(p.q_out) + t * p.q_out_token + r * p.q_out_head
                       : static_cast<T*>(p.k_out) + t * p.k_out_token + (r - p.H) * p.k_out_head;
#pragma unroll
      for (int k = 0; k < KU; ++k) {
        if (k >= have) continue;
        C a, b;
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
          a.e[e] = Elem<DT>::put(fmaf(-v[k][e], c, rr * (w[k][e] * d[k][e])));
          b.e[e] = Elem<DT>::put(fmaf(-v[k][VEC + e], c, rr * (w[k][VEC + e] * d[k][VEC + e])));
        }
        *reinterpret_cast<C*>(dst + oa[k]) = a;
        *reinterpret_cast<C*>(dst + ob[k]) = b;
      }
    }
  }
  if (!p.part) return;
  // the groups of a warp, then the warps, per kind of row
  __shared__ float s_dw[kRopeThreads / 32][512];
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
#pragma unroll
  for (int kd = 0; kd < 2; ++kd) {
    __syncthreads();
#pragma unroll
    for (int k = 0; k < KU; ++k)
#pragma unroll
      for (int e = 0; e < 2 * VEC; ++e) {
        float s = dw[kd][k][e];
        for (int o = ln; o < 32; o *= 2) s += __shfl_xor_sync(kAll, s, o);
        if (lane < ln && k < have) s_dw[warp][(e < VEC ? oa[k] : ob[k] - VEC) + e] = s;
      }
    __syncthreads();
    for (int i = threadIdx.x; i < p.d; i += kRopeThreads) {
      float s = 0.f;
#pragma unroll
      for (int x = 0; x < kRopeThreads / 32; ++x) s += s_dw[x][i];
      p.part[(static_cast<size_t>(blockIdx.x) * 2 + kd) * p.d + i] = s;
    }
  }
}

// Column c of the CTAs' partial sums [ctas][2 d]: 32 columns and 32 shares of the CTAs per CTA.
__global__ void __launch_bounds__(1024)
    norm_rope_sum_kernel(const float* part, int ctas, int d, float* dq_weight, float* dk_weight) {
  __shared__ float s[32][33];
  const int lane = threadIdx.x % 32, share = threadIdx.x / 32, c = blockIdx.x * 32 + lane;
  float x = 0.f;
  if (c < 2 * d)
    for (int i = share; i < ctas; i += 32) x += part[static_cast<size_t>(i) * 2 * d + c];
  s[share][lane] = x;
  __syncthreads();
  x = s[lane][share];  // lane: share; share: column
#pragma unroll
  for (int o = 16; o > 0; o /= 2) x += __shfl_xor_sync(kAll, x, o);
  const int col = blockIdx.x * 32 + share;
  if (lane == 0 && col < 2 * d) {
    float* out = col < d ? dq_weight : dk_weight;
    if (out) out[col < d ? col : col - d] = x;
  }
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

template <int DT, int VEC, int KU, int MODE>
cudaError_t launch_v(const NormRopeParams& p, bool half_style, int sms, cudaStream_t stream) {
  // Tokens per CTA: one while that leaves SMs without work (a decode step), four for a prompt.
  const int tok = p.T >= 16LL * sms ? 4 : 1;
  const int ln = lanes_of(p.d / (2 * VEC), KU);
  const size_t smem = static_cast<size_t>(p.rot / 2) * (tok * sizeof(float2) + sizeof(uint64_t) + 1);
  const int64_t grid = (p.T + tok - 1) / tok;
  if (grid > 0x7fffffff) return cudaErrorInvalidConfiguration;
  auto* k = half_style ? norm_rope_kernel<DT, VEC, KU, true, MODE>
                       : norm_rope_kernel<DT, VEC, KU, false, MODE>;
  k<<<static_cast<unsigned>(grid), kRopeThreads, smem, stream>>>(p, tok, ln);
  return cudaGetLastError();
}
template <int DT, int VEC, int KU>
cudaError_t launch_bwd_v(const NormRopeParams& p, bool half_style, int sms, cudaStream_t stream) {
  const int tok = p.T >= 16LL * sms ? 4 : 1;
  const int ln = lanes_of(p.d / (2 * VEC), KU);
  const size_t smem = static_cast<size_t>(p.rot / 2) * (tok * sizeof(float2) + sizeof(uint64_t) + 1);
  const int64_t batches = (p.T + tok - 1) / tok;
  const int64_t most = 2 * sms < kNormCtas ? 2 * sms : kNormCtas;
  const int grid = static_cast<int>(batches < most ? batches : most);
  auto* k = half_style ? norm_rope_bwd_kernel<DT, VEC, KU, true>
                       : norm_rope_bwd_kernel<DT, VEC, KU, false>;
  k<<<grid, kRopeThreads, smem, stream>>>(p, tok, ln);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || !p.part) return e;
  norm_rope_sum_kernel<<<(2 * p.d + 31) / 32, 1024, 0, stream>>>(p.part, grid, p.d, p.dq_weight,
                                                                 p.dk_weight);
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
