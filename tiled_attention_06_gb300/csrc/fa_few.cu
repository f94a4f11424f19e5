// Attention of a few new rows over a paged cache with grouped heads, for sm_103a: a decode
// step, or a couple of drafted tokens. The rows of a sequence and K/V head are its tokens times
// the G query heads that share the head (row r: token r / G, head r % G); at most 16.
//
// Bound by reading K and V once: 4 d bytes per key and K/V head against 4 d G multiply-adds per
// token, which the FP32 pipes cannot keep up with from G = 4 or so, hence warp-level tensor-core
// MMAs (m16n8k16, whose 16 rows fit; at 6.2 TB/s their pipe is 16 % busy). With 32 or 64 rows
// this form was bound by the latency of its MMAs (40 rows over 84,000 keys x 4 heads: 49 us
// where the memory needs 26), and the 128-row tiles of fa_varlen.cu take over.
//
// few_kernel, two CTAs per SM, each four compute warps and a TMA warp. The 64-key tiles of all
// (sequence, K/V head) pairs are numbered end to end and CTA x takes an equal run of them, so
// ragged lengths cost no balance. A run's piece of one pair is a segment: a whole pair is written
// to o, a piece to the workspace. A warp takes 16 keys of every tile and keeps its own running
// maximum, sum and output in registers; the four are joined through shared memory at the end of
// a segment.
// 32 sequences of 110,000 keys in all, 32/8 heads of 128, fp16: 79 to 84 us, 6.1 TB/s (the join
// 4 more; the cache's bytes alone take 72.6 us at the measured copy rate).
// few_merge_kernel joins the pieces of each pair in the order of the keys; the CTA that holds a
// pair's first piece leaves word of where the others are.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <climits>
#include <cstdint>

#include "fa_plan.h"
#include "fa_ptx.cuh"
#include "fa_varlen.h"

namespace fa {
namespace {

constexpr int BK = 64;              // keys per tile
constexpr int ROWS = kFewRows;      // rows of a warp's tile
constexpr int NW = 4;               // compute warps; the next one loads
constexpr int kCompute = 32 * NW;
constexpr int kThreads = kCompute + 32;
constexpr float kTau = 8.0f;        // lazy-rescale threshold, log2 units

template <int D>
struct Cfg {
  static constexpr int KCH = D / 64;
  static constexpr int TILE = BK * D * 2;    // K or V of one tile
  static constexpr int COMB = 2 * 16 * D * 4;  // two warps' outputs
  static constexpr int STATES = 4 * 16 * 2 * 4;  // (m, l) of four warps
  static constexpr int BARS = 256;
  // two CTAs share an SM's 228 KB, 1 KB of it taken per CTA
  static constexpr int BUDGET = 233472 / 2 - 1024;
  static constexpr int FIT = (BUDGET - COMB - STATES - BARS) / (2 * TILE);
  static constexpr int NST = FIT > 8 ? 8 : FIT;
  static constexpr int SMEM = NST * 2 * TILE + COMB + STATES + BARS;
  static_assert(NST >= 3, "too few stages");
};

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
__device__ __forceinline__ void compute_sync() {
  asm volatile("bar.sync 1, %0;" ::"n"(kCompute) : "memory");
}

// One sequence: its rows, keys and the tiles that the mask lets its queries see.
struct FewSeq {
  int q0, n, sk, qpos, tiles;
  Range rg;
};
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

// Sums over the CTA's first 128 threads of each thread's contiguous share of the sequences.
struct Totals {
  int64_t before, mine, all;  // tiles before this thread's share, in it, of every sequence
  int b0, b1;                 // the share
};
__device__ __forceinline__ Totals tile_totals(const FewParams& p, int64_t* scratch) {
  Totals t{0, 0, 0, 0, 0};
  const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32;
  int64_t x = 0;
  if (tid < kCompute) {
    const int per = (p.B + kCompute - 1) / kCompute;
    t.b0 = min(p.B, tid * per);
    t.b1 = min(p.B, t.b0 + per);
    for (int b = t.b0; b < t.b1; ++b) x += few_seq(p, b, blockIdx.x == 0).tiles;
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

template <int D, bool BF16>
__global__ void __launch_bounds__(kThreads, 2)
    few_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
               const __grid_constant__ FewParams p) {
  using C = Cfg<D>;
  constexpr int KPW = BK / NW;    // keys of a warp per tile
  constexpr int NT = KPW / 8;     // 8-key columns of S
  constexpr int NO = D / 8;       // 8-element columns of O
  extern __shared__ __align__(1024) uint8_t smem[];
  const uint32_t base = smem_u32(smem);
  float* comb = reinterpret_cast<float*>(smem + C::NST * 2 * C::TILE);
  float* states = reinterpret_cast<float*>(smem + C::NST * 2 * C::TILE + C::COMB);
  Bars* bars =
      reinterpret_cast<Bars*>(smem + C::NST * 2 * C::TILE + C::COMB + C::STATES);
  auto B = [&](uint64_t& x) { return smem_u32(&x); };
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  // whatever ends this CTA early, the joining kernel finds no piece of it
  if (threadIdx.x == 0) p.heads[blockIdx.x] = FewHead{0, 0, 0, 0};
  if (base & 1023u) {  // the swizzle needs the stages on 1024-byte boundaries
    if (threadIdx.x == 0) atomicOr(p.m.status, FA_DEV_SMEM_BASE);
    return;
  }
  if (threadIdx.x == 0) {
    for (int i = 0; i < C::NST; ++i) {
      mbar_init(B(bars->full[i]), 1);
      mbar_init(B(bars->empty[i]), NW);
    }
    bars->abort = 0;
    mbar_fence_init();
  }
  if (warp == NW && lane == 0) {
    tma_prefetch_desc(&tmK);
    tma_prefetch_desc(&tmV);
  }
  const Totals tot = tile_totals(p, bars->sum);
  const int64_t all = tot.all * p.Hkv;
  const int used = ctas_used(all, gridDim.x);
  const bool idle = static_cast<int>(blockIdx.x) >= used || all == 0;
  if (threadIdx.x == 0) {
    bars->all = all;
    bars->used = used;
  }
  const int64_t begin = idle ? 0 : all * blockIdx.x / used;
  const int64_t end = idle ? 0 : all * (blockIdx.x + 1) / used;
  // the thread whose share holds the first tile finds its sequence
  if (!idle && threadIdx.x < kCompute && begin >= tot.before * p.Hkv &&
      begin < (tot.before + tot.mine) * p.Hkv) {
    int64_t at = tot.before * p.Hkv;
    for (int b = tot.b0; b < tot.b1; ++b) {
      const int64_t n = static_cast<int64_t>(few_seq(p, b, false).tiles) * p.Hkv;
      if (begin < at + n) {
        bars->first[0] = b;
        bars->first[1] = static_cast<int>(begin - at);
        break;
      }
      at += n;
    }
  }
  if (blockIdx.x == 0 && threadIdx.x < kCompute) {  // chunks that see no key at all
    for (int b = tot.b0; b < tot.b1; ++b) {
      const FewSeq s = few_seq(p, b, false);
      if (s.tiles > 0) continue;
      for (int t = s.q0; t < s.q0 + s.n; ++t) {
        uint4* dst = reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.o) + t * p.o_token);
        for (int i = 0; i < p.H * D / 8; ++i) dst[i] = make_uint4(0, 0, 0, 0);
        for (int h = 0; h < p.H && p.lse; ++h) p.lse[static_cast<size_t>(t) * p.H + h] = -INFINITY;
      }
    }
  }
  __syncthreads();
  if (begin >= end) return;  // uniform: no barrier is used from here
  Walk w;
  w.b = bars->first[0];
  w.s = few_seq(p, w.b, false);
  w.kvh = bars->first[1] / w.s.tiles;
  w.j = bars->first[1] - w.kvh * w.s.tiles;
  w.left = static_cast<int>(end - begin);
  // step to the segment after one of `done` tiles
  auto advance = [&](int done) {
    w.left -= done;
    w.j = 0;
    if (++w.kvh < p.Hkv || w.left <= 0) return;
    w.kvh = 0;
    do {
      w.s = few_seq(p, ++w.b, false);
    } while (w.s.tiles == 0);  // ends: `left` tiles lie ahead
  };
  const WaitCtx wc{&bars->abort, p.m.status, p.m.timeout_ns};

  if (warp == NW) {
    // -------------------------------------------------------------- TMA
    // lane = (K or V, 64-element region of d, box of the tile)
    const bool leader = elect_one();
    const int per_tile = BK / p.box;
    const int kv = lane / (C::KCH * per_tile), c = (lane / per_tile) % C::KCH, bx = lane % per_tile;
    uint32_t pos = 0, fills[8] = {0, 0, 0, 0, 0, 0, 0, 0};
    bool ok = true;
    while (w.left > 0 && ok) {
      const int cnt = min(w.left, w.s.tiles - w.j);
      for (int j = w.j; j < w.j + cnt && ok; ++j, ++pos) {
        const int n0 = tile_at(w.s.rg, j) * BK;
        const int boxes = (min(BK, w.s.sk - n0) + p.box - 1) / p.box;
        int y = 0, z = 0;
        if (kv < 2 && bx < boxes) {
          const int row = n0 + bx * p.box, lp = row / p.page_size;
          int phys = p.block_table[static_cast<size_t>(w.b) * p.max_pages + lp];
          if (phys < 0 || phys >= p.num_pages) {
            atomicOr(p.m.status, FA_DEV_BAD_PAGE);
            phys = 0;
          }
          y = row - lp * p.page_size;
          z = phys * p.Hkv + w.kvh;
        }
        const int st = pos % C::NST;
        const uint32_t use = pos / C::NST;
        if (!(ok = mbar_wait(B(bars->empty[st]), (use & 1) ^ 1, wc))) break;
        if (leader) mbar_arrive_expect_tx(B(bars->full[st]), boxes * p.box * C::KCH * 256);
        __syncwarp();
        if (kv < 2 && bx < boxes)
          tma_load_3d(base + (2 * st + kv) * C::TILE + c * (BK * 128) + bx * p.box * 128,
                      kv ? (const void*)&tmV : (const void*)&tmK, B(bars->full[st]), c * 64, y, z);
        __syncwarp();
        fills[st] = use + 1;
      }
      advance(cnt);
    }
    if (!ok) {  // every load issued lands before the CTA exits
      volatile uint32_t zero = 0;
      WaitCtx quiet = wc;
      quiet.abort = &zero;
      for (int i = 0; i < C::NST; ++i)
        if (fills[i] > 0) mbar_wait(B(bars->full[i]), (fills[i] - 1) & 1, quiet);
    }
    return;
  }
  // ---------------------------------------------------------------- compute
  const int kw = warp, r0 = lane / 4;  // key group; this thread's rows are r0 and r0 + 8
  const int cq = lane % 4;
  uint32_t pos = 0;
  bool ok = true;
  while (w.left > 0) {
    const int cnt = min(w.left, w.s.tiles - w.j);
    const int rows = w.s.n * p.G;
    // Q fragments straight from global memory (rows past the chunk are zero)
    uint32_t qf[D / 16][4];
    int tok[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int r = r0 + 8 * i;
      tok[i] = r / p.G;
      const uint16_t* src = static_cast<const uint16_t*>(p.q) +
                            static_cast<int64_t>(w.s.q0 + tok[i]) * p.q_token +
                            (w.kvh * p.G + r - tok[i] * p.G) * D + 2 * cq;
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk) {
        qf[kk][i] = r < rows ? *reinterpret_cast<const uint32_t*>(src + 16 * kk) : 0u;
        qf[kk][2 + i] = r < rows ? *reinterpret_cast<const uint32_t*>(src + 16 * kk + 8) : 0u;
      }
    }
    float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f}, o[NO][4];
#pragma unroll
    for (int i = 0; i < NO; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[i][e] = 0.f;
    for (int j = w.j; j < w.j + cnt; ++j, ++pos) {
      const int n0 = tile_at(w.s.rg, j) * BK;
      const int st = pos % C::NST;
      // a warp that gives up still meets the others at the joins (its results are void)
      ok = ok && mbar_wait(B(bars->full[st]), (pos / C::NST) & 1, wc);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) continue;
      const uint32_t sK = base + 2 * st * C::TILE, sV = sK + C::TILE;
      const int live = w.s.sk - n0;
      float s[NT][4];
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int e = 0; e < 4; ++e) s[t][e] = 0.f;
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk) {
#pragma unroll
        for (int t = 0; t < NT; t += 2) {
          const int key = kw * KPW + 8 * t + (lane / 16) * 8 + lane % 8;
          const int ch = 2 * kk + (lane / 8) % 2;
          uint32_t kf[4];
          ldsm4(sK + (ch / 8) * (BK * 128) + key * 128 + (((ch % 8) ^ (key & 7)) << 4), kf);
          mma<BF16>(s[t], qf[kk], kf[0], kf[1]);
          mma<BF16>(s[t + 1], qf[kk], kf[2], kf[3]);
        }
      }
      // hidden keys to -inf where some row does not see the whole tile
      const int lo_pos = w.s.qpos, hi_pos = w.s.qpos + w.s.n - 1;
      bool full = n0 + BK <= w.s.sk;
      if (p.m.mask_mode != FA_MASK_NONE) {
        if (p.m.mask_mode == FA_MASK_CAUSAL || p.m.mask_mode == FA_MASK_CAUSAL_WINDOW)
          full = full && n0 + BK - 1 <= lo_pos;
        if (p.m.mask_mode == FA_MASK_CAUSAL_WINDOW)
          full = full && (n0 + BK <= p.m.n_global || hi_pos - max(n0, p.m.n_global) < p.m.window);
        if (p.m.mask_mode == FA_MASK_BAND)
          full = full && static_cast<long long>(hi_pos) - n0 <= p.m.window &&
                 static_cast<long long>(n0 + BK - 1) - lo_pos <= p.m.window;
        if (p.m.mask_mode == FA_MASK_PREFIX_LM)
          full = full && (n0 + BK <= p.m.n_global || n0 + BK - 1 <= lo_pos);
      }
      if (!full) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          // keys of the tile that the row sees: up to lim, and from lo on or below gl
          const long long at = static_cast<long long>(w.s.qpos) + tok[i] - n0;
          const int last = w.s.sk - 1 - n0, wide = p.m.window;
          long long hi = at, from = -1;
          int gl = 0;
          if (p.m.mask_mode == FA_MASK_NONE) hi = BK;
          if (p.m.mask_mode == FA_MASK_CAUSAL_WINDOW) {
            from = at - wide + 1;
            gl = p.m.n_global - n0;
          }
          if (p.m.mask_mode == FA_MASK_BAND) {
            hi = at + wide;
            from = at - wide;
          }
          if (p.m.mask_mode == FA_MASK_PREFIX_LM)
            hi = max(at, static_cast<long long>(p.m.n_global) - 1 - n0);
          const int lim = min(static_cast<int>(max(-1ll, min(hi, static_cast<long long>(BK)))), last);
          const int lo = static_cast<int>(max(-1ll, min(from, static_cast<long long>(BK))));
#pragma unroll
          for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const int key = kw * KPW + 8 * t + 2 * cq + e;
              if (!(key <= lim && (key >= lo || key < gl))) s[t][2 * i + e] = -INFINITY;
            }
        }
      }
      // running maximum (a row is shared by four lanes), lazy rescale, P
      bool need = false;
      float mn[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        float mx = -INFINITY;
#pragma unroll
        for (int t = 0; t < NT; ++t) mx = max3f(mx, s[t][2 * i], s[t][2 * i + 1]);
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
        mn[i] = fmaxf(m[i], mx * p.m.sl2);
        need = need || (m[i] != -INFINITY && mn[i] > m[i] + kTau);
        if (m[i] == -INFINITY) m[i] = mn[i];
      }
      if (__any_sync(0xffffffffu, need)) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const bool move = mn[i] > m[i] + kTau;
          const float a = move ? ex2_approx(m[i] - mn[i]) : 1.f;
          if (move) m[i] = mn[i];
          l[i] *= a;
#pragma unroll
          for (int t = 0; t < NO; ++t) {
            o[t][2 * i] *= a;
            o[t][2 * i + 1] *= a;
          }
        }
      }
      uint32_t pf[NT][2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const float mu = m[i] == -INFINITY ? 0.f : m[i];
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          const float a = ex2_approx(fmaf(s[t][2 * i], p.m.sl2, -mu));
          const float b = ex2_approx(fmaf(s[t][2 * i + 1], p.m.sl2, -mu));
          l[i] += a + b;
          pf[t][i] = BF16 ? cvt_pack_bf16(a, b) : cvt_pack_f16(a, b);
        }
      }
      if (live < BK) {  // rows of V behind the last key: 0 times what they hold may not be 0
        for (int i = lane; i < KPW * 8 * C::KCH; i += 32) {
          const int key = kw * KPW + (i / 8) % KPW;
          if (key >= live)
            st_shared_v4(sV + (i / (8 * KPW)) * (BK * 128) + key * 128 + (i % 8) * 16, 0, 0, 0, 0);
        }
        fence_proxy_async_smem();  // before the slot's next load
        __syncwarp();
      }
#pragma unroll
      for (int kk = 0; kk < NT / 2; ++kk) {  // 16 keys
        const uint32_t pa[4] = {pf[2 * kk][0], pf[2 * kk][1], pf[2 * kk + 1][0], pf[2 * kk + 1][1]};
        const int key = kw * KPW + 16 * kk + ((lane / 8) % 2) * 8 + lane % 8;
#pragma unroll
        for (int t = 0; t < NO; t += 2) {
          const int ch = t + lane / 16;
          uint32_t vf[4];
          ldsm4_t(sV + (ch / 8) * (BK * 128) + key * 128 + (((ch % 8) ^ (key & 7)) << 4), vf);
          mma<BF16>(o[t], pa, vf[0], vf[1]);
          mma<BF16>(o[t + 1], pa, vf[2], vf[3]);
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(B(bars->empty[st]));
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      l[i] += __shfl_xor_sync(0xffffffffu, l[i], 1);
      l[i] += __shfl_xor_sync(0xffffffffu, l[i], 2);
    }
    // join the key groups: the upper half hands its state to the lower, until one is left
#pragma unroll
    for (int half = NW / 2; half >= 1; half /= 2) {
      if (kw >= half && kw < 2 * half) {
        float* dst = comb + (kw - half) * 16 * D;
        float* sd = states + (kw - half) * 32;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int r = r0 + 8 * i;
#pragma unroll
          for (int t = 0; t < NO; ++t)
            *reinterpret_cast<float2*>(dst + r * D + 8 * t + 2 * cq) =
                make_float2(o[t][2 * i], o[t][2 * i + 1]);
          if (cq == 0) {
            sd[r] = m[i];
            sd[16 + r] = l[i];
          }
        }
      }
      compute_sync();
      if (kw < half) {
        const float* src = comb + kw * 16 * D;
        const float* sd = states + kw * 32;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int r = r0 + 8 * i;
          const float m2 = sd[r], M = fmaxf(m[i], m2), mu = M == -INFINITY ? 0.f : M;
          const float a = ex2_approx(m[i] - mu), b = ex2_approx(m2 - mu);
          l[i] = l[i] * a + sd[16 + r] * b;
          m[i] = M;
#pragma unroll
          for (int t = 0; t < NO; ++t) {
            const float2 v = *reinterpret_cast<const float2*>(src + r * D + 8 * t + 2 * cq);
            o[t][2 * i] = o[t][2 * i] * a + v.x * b;
            o[t][2 * i + 1] = o[t][2 * i + 1] * a + v.y * b;
          }
        }
      }
      compute_sync();
    }
    if (kw == 0) {
      const bool whole = w.j == 0 && cnt == w.s.tiles;
      // a piece that starts its pair goes to slot 2x + 1, one that continues it to slot 2x
      const int slot = 2 * blockIdx.x + (w.j == 0 ? 1 : 0);
      const int nslots = 2 * gridDim.x;
      if (!whole && w.j == 0 && threadIdx.x == 0) {
        // the piece that starts a pair says where the rest is: CTAs on to that of its last tile
        const int64_t n = bars->all, own_end = n * (blockIdx.x + 1) / bars->used;
        const int64_t last = own_end - w.left + w.s.tiles - 1;
        int x = blockIdx.x + 1;
        while (n * (x + 1) / bars->used <= last) ++x;
        p.heads[blockIdx.x] = FewHead{w.s.q0, rows, w.kvh, x};
      }
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int r = r0 + 8 * i;
        if (r >= rows) continue;
        const int head = w.kvh * p.G + r - tok[i] * p.G;
        if (whole) {
          const float inv = l[i] != 0.f ? 1.f / l[i] : 0.f;
          uint16_t* dst = static_cast<uint16_t*>(p.o) +
                          static_cast<int64_t>(w.s.q0 + tok[i]) * p.o_token + head * D + 2 * cq;
#pragma unroll
          for (int t = 0; t < NO; ++t) {
            const float a = o[t][2 * i] * inv, b = o[t][2 * i + 1] * inv;
            *reinterpret_cast<uint32_t*>(dst + 8 * t) = BF16 ? cvt_pack_bf16(a, b) : cvt_pack_f16(a, b);
          }
          if (cq == 0 && p.lse)
            p.lse[static_cast<size_t>(w.s.q0 + tok[i]) * p.H + head] = lse_of(m[i], l[i]);
        } else {
          float* dst = p.part + (static_cast<size_t>(slot) * ROWS + r) * D + 2 * cq;
#pragma unroll
          for (int t = 0; t < NO; ++t)
            *reinterpret_cast<float2*>(dst + 8 * t) = make_float2(o[t][2 * i], o[t][2 * i + 1]);
          if (cq == 0) {
            float* ml = p.part + static_cast<size_t>(nslots) * ROWS * D;
            ml[slot * ROWS + r] = m[i];
            ml[(nslots + slot) * ROWS + r] = l[i];
          }
        }
      }
    }
    advance(cnt);
  }
}

// CTA (x, y): row y of the pair whose first piece CTA x of few_kernel holds. A warp's lanes hold
// the pieces' maxima and sums, so the weights are known before the outputs are read; the four
// warps take every fourth piece.
template <int D, bool BF16>
__global__ void __launch_bounds__(kCompute) few_merge_kernel(const FewParams p) {
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

template <int D, bool BF16>
cudaError_t launch_t(const FewLaunch& L, cudaStream_t stream) {
  const int grid = 2 * L.sms < kFewMaxCtas ? 2 * L.sms : kFewMaxCtas;
  auto* k = few_kernel<D, BF16>;
  constexpr int smem = Cfg<D>::SMEM;
  cudaError_t e = prepare_kernel<few_kernel<D, BF16>>(smem);
  if (e != cudaSuccess) return e;
  k<<<grid, kThreads, smem, stream>>>(L.tmK, L.tmV, L.p);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  const int rows = L.p.max_q * L.p.G;
  few_merge_kernel<D, BF16><<<dim3(grid, rows < 1 ? 1 : rows), kCompute, 0, stream>>>(L.p);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_few(const FewLaunch& L, int D, bool bf16, cudaStream_t stream) {
  if (D == 128) return bf16 ? launch_t<128, true>(L, stream) : launch_t<128, false>(L, stream);
  return bf16 ? launch_t<64, true>(L, stream) : launch_t<64, false>(L, stream);
}

}  // namespace fa
