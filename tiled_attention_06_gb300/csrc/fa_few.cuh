// What the kernels for a few rows over a paged cache share (fa_few.cu, fa_few8.cu): the numbering of
// all sequences' key tiles, a CTA's run of them, warp-level products, and the joining of pieces.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <climits>
#include <cstdint>

#include "fa_plan.h"
#include "fa_ptx.cuh"
#include "fa_varlen.h"

namespace fa {
namespace {

constexpr int NW = 4;               // compute warps; the next one loads
constexpr int kCompute = 32 * NW;
constexpr int kThreads = kCompute + 32;
constexpr float kTau = 8.0f;        // lazy-rescale threshold, log2 units

struct Bars {
  uint64_t full[8], empty[8];
  int64_t sum[4];   // scratch of tile_totals
  int64_t all;      // tiles of the call, and the CTAs that share them
  int used;
  int first[2];     // sequence of the CTA's first tile, tile within it (all K/V heads)
  uint32_t abort;
};
static_assert(sizeof(Bars) <= 256, "barrier block over its reserve");

__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t* r) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm4_t(uint32_t addr, uint32_t* r) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
// c (16 x 8, FP32) += a (16 x 16) b (16 x 8)
template <bool BF16>
__device__ __forceinline__ void mma(float* c, const uint32_t* a, uint32_t b0, uint32_t b1) {
  if constexpr (BF16)
    asm(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
        "{%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
        "{%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// One sequence: its rows, keys and the tiles that the mask lets its queries see.
struct FewSeq {
  int q0, n, sk, qpos, tiles;
  Range rg;
};
// BK: keys of a tile; TREE: the call may have a tree.
template <int BK, bool TREE>
__device__ __forceinline__ FewSeq few_seq(const FewParams& p, int b, bool report) {
  FewSeq s;
  const int a = p.cu_q[b], e = p.cu_q[b + 1], cap = p.page_size * p.max_pages;
  int sk = p.ctx[b];
  bool bad = a < 0 || e < a || e > p.total_q;
  s.q0 = bad ? 0 : a;
  const int n = bad ? 0 : e - a;
  bad = bad || sk < 0 || sk > cap || n > p.max_q;
  sk = sk < 0 ? 0 : min(sk, cap);
  if (bad && report) atomicOr(p.m.status, FA_DEV_BAD_PAGE);
  s.n = min(n, p.max_q);
  s.sk = sk;
  s.qpos = sk - n;
  PrefillParams f;  // ranges by key position: as many queries as keys
  f.mask_mode = p.m.mask_mode;
  if (TREE && f.mask_mode == FA_MASK_TREE) f.mask_mode = FA_MASK_NONE;
  f.window = p.m.window;
  f.n_global = p.m.n_global;
  f.Sq = sk;
  s.rg = key_range(s.qpos, s.qpos + s.n, BK, sk, f, 0);
  s.tiles = range_count(s.rg);
  return s;
}
__device__ __forceinline__ int tile_at(const Range& r, int j) {
  return j < r.a_end ? j : r.b_start + (j - r.a_end);
}

// Sums over the CTA's first 128 threads of each thread's contiguous share of the sequences, of units:
// a sequence's tiles and, where it has any, EXTRA more.
struct Totals {
  int64_t before, mine, all;  // units before this thread's share, in it, of every sequence
  int b0, b1;                 // the share
};
template <int BK, bool TREE, int EXTRA>
__device__ __forceinline__ Totals tile_totals(const FewParams& p, int64_t* scratch) {
  Totals t{0, 0, 0, 0, 0};
  const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32;
  int64_t x = 0;
  if (tid < kCompute) {
    const int per = (p.B + kCompute - 1) / kCompute;
    t.b0 = min(p.B, tid * per);
    t.b1 = min(p.B, t.b0 + per);
    for (int b = t.b0; b < t.b1; ++b) {
      const int tiles = few_seq<BK, TREE>(p, b, blockIdx.x == 0).tiles;
      x += EXTRA && tiles ? tiles + EXTRA : tiles;
    }
    t.mine = x;
    for (int o = 1; o < 32; o *= 2) {
      const int64_t y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    if (lane == 31) scratch[warp] = x;
  }
  __syncthreads();
  for (int w = 0; w < kCompute / 32; ++w) {
    if (w < warp) t.before += scratch[w];
    t.all += scratch[w];
  }
  t.before += x - t.mine;
  return t;
}

// CTAs that share the tiles: two at least for each (a tile is about 1.3 us of one CTA's share
// of the bandwidth, a merge of many short pieces costs more than it spreads).
__device__ __forceinline__ int ctas_used(int64_t tiles, int grid) {
  const int64_t want = (tiles + 1) / 2;
  return static_cast<int>(want < grid ? (want < 1 ? 1 : want) : grid);
}

// A walk over the tiles [t, end) of this CTA: one segment after the other.
struct Walk {
  int b, kvh, j, left;
  FewSeq s;
};

// CTA (x, y): row y of the pair whose first piece CTA x of few_kernel holds. A warp's lanes hold
// the pieces' maxima and sums, so the weights are known before the outputs are read; the four
// warps take every fourth piece.
// EARLY: launched while the kernel before it runs (programmatic stream serialization), it waits here.
template <int D, bool BF16, int ROWS, bool EARLY>
__global__ void __launch_bounds__(kCompute) few_merge_kernel(const FewParams p) {
  if constexpr (EARLY) asm volatile("griddepcontrol.wait;" ::: "memory");
  constexpr int E = D / 32;
  __shared__ float s_acc[4][D];
  const int x0 = blockIdx.x, nslots = 2 * gridDim.x, r = blockIdx.y;
  const FewHead hd = p.heads[x0];
  if (r >= hd.rows) return;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const float* ml = p.part + static_cast<size_t>(nslots) * ROWS * D;
  auto slot_of = [&](int x) { return 2 * x + (x == x0 ? 1 : 0); };
  // maximum and sum over the pieces, one per lane; loads before their uses throughout
  float M = -INFINITY, L = 0.f;
  for (int x1 = x0; x1 <= hd.last; x1 += 32) {
    const int x = x1 + lane;
    float m = -INFINITY, l = 0.f;
    if (x <= hd.last) {
      m = ml[slot_of(x) * ROWS + r];
      l = ml[(nslots + slot_of(x)) * ROWS + r];
    }
    float mx = fmaxf(M, m);
#pragma unroll
    for (int o = 16; o > 0; o /= 2) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
    const float mu = mx == -INFINITY ? 0.f : mx;
    l *= ex2_approx(m - mu);
#pragma unroll
    for (int o = 16; o > 0; o /= 2) l += __shfl_xor_sync(0xffffffffu, l, o);
    L = L * ex2_approx(M - mu) + l;
    M = mx;
  }
  const float mu = M == -INFINITY ? 0.f : M;
  float acc[E];
#pragma unroll
  for (int e = 0; e < E; ++e) acc[e] = 0.f;
  constexpr int N = 6;  // pieces of this warp in flight
  for (int x1 = x0 + warp; x1 <= hd.last; x1 += 4 * N) {
    float m[N], v[N][E];
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int x = x1 + 4 * i;
      m[i] = -INFINITY;
#pragma unroll
      for (int e = 0; e < E; ++e) v[i][e] = 0.f;
      if (x <= hd.last) {
        const int s = slot_of(x);
        m[i] = ml[s * ROWS + r];
        const float* src = p.part + (static_cast<size_t>(s) * ROWS + r) * D + lane * E;
#pragma unroll
        for (int e = 0; e < E; ++e) v[i][e] = src[e];
      }
    }
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const float w = ex2_approx(m[i] - mu);
#pragma unroll
      for (int e = 0; e < E; ++e) acc[e] = fmaf(w, v[i][e], acc[e]);
    }
  }
#pragma unroll
  for (int e = 0; e < E; ++e) s_acc[warp][lane * E + e] = acc[e];
  __syncthreads();
  const int tok = r / p.G, h = hd.kvh * p.G + r - tok * p.G;
  const float inv = L != 0.f ? 1.f / L : 0.f;
  uint16_t* out =
      static_cast<uint16_t*>(p.o) + static_cast<int64_t>(hd.q0 + tok) * p.o_token + h * D;
  for (int e = 2 * threadIdx.x; e < D; e += 2 * kCompute) {
    float a = 0.f, c = 0.f;
    for (int k = 0; k < 4; ++k) {
      a += s_acc[k][e];
      c += s_acc[k][e + 1];
    }
    *reinterpret_cast<uint32_t*>(out + e) =
        BF16 ? cvt_pack_bf16(a * inv, c * inv) : cvt_pack_f16(a * inv, c * inv);
  }
  if (threadIdx.x == 0 && p.lse)
    p.lse[static_cast<size_t>(hd.q0 + tok) * p.H + h] = lse_of(M, L);
}

}  // namespace
}  // namespace fa
