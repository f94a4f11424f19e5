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
#include <cstdint>

#include "fa_few.cuh"

namespace fa {
namespace {

constexpr int BK = 64;              // keys per tile
constexpr int ROWS = kFewRows;      // rows of a warp's tile

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

__device__ __forceinline__ void compute_sync() {
  asm volatile("bar.sync 1, %0;" ::"n"(kCompute) : "memory");
}

// TREE: masks from the caller (FA_MASK_TREE); a form of its own, so that the other carries nothing of it.
template <int D, bool BF16, bool TREE>
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
  const Totals tot = tile_totals<BK, TREE, 0>(p, bars->sum);
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
      const int64_t n = static_cast<int64_t>(few_seq<BK, TREE>(p, b, false).tiles) * p.Hkv;
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
      const FewSeq s = few_seq<BK, TREE>(p, b, false);
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
  w.s = few_seq<BK, TREE>(p, w.b, false);
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
      w.s = few_seq<BK, TREE>(p, ++w.b, false);
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
        if (TREE && p.m.mask_mode == FA_MASK_TREE) full = full && n0 + BK <= lo_pos;
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
          uint32_t seen = ~0u;  // a tree's bits for the warp's keys
          if (TREE && p.m.mask_mode == FA_MASK_TREE) {
            hi = BK;
            if (tok[i] < w.s.n)
              seen = tree_bits(p.tree + static_cast<size_t>(w.s.q0 + tok[i]) * p.tree_words,
                               p.tree_words, n0 + kw * KPW - w.s.qpos);
          }
          const int lim = min(static_cast<int>(max(-1ll, min(hi, static_cast<long long>(BK)))), last);
          const int lo = static_cast<int>(max(-1ll, min(from, static_cast<long long>(BK))));
#pragma unroll
          for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const int key = kw * KPW + 8 * t + 2 * cq + e;
              if (!(key <= lim && (key >= lo || key < gl))) s[t][2 * i + e] = -INFINITY;
              if (TREE && !((seen >> (8 * t + 2 * cq + e)) & 1)) s[t][2 * i + e] = -INFINITY;
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

template <int D, bool BF16, bool TREE>
cudaError_t launch_t(const FewLaunch& L, cudaStream_t stream) {
  const int grid = 2 * L.sms < kFewMaxCtas ? 2 * L.sms : kFewMaxCtas;
  auto* k = few_kernel<D, BF16, TREE>;
  constexpr int smem = Cfg<D>::SMEM;
  cudaError_t e = prepare_kernel<few_kernel<D, BF16, TREE>>(smem);
  if (e != cudaSuccess) return e;
  k<<<grid, kThreads, smem, stream>>>(L.tmK, L.tmV, L.p);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  const int rows = L.p.max_q * L.p.G;
  few_merge_kernel<D, BF16, ROWS, false>
      <<<dim3(grid, rows < 1 ? 1 : rows), kCompute, 0, stream>>>(L.p);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_few(const FewLaunch& L, int D, bool bf16, cudaStream_t stream) {
  const bool tree = L.p.m.mask_mode == FA_MASK_TREE;
  if (D == 128)
    return bf16 ? (tree ? launch_t<128, true, true>(L, stream) : launch_t<128, true, false>(L, stream))
                : (tree ? launch_t<128, false, true>(L, stream) : launch_t<128, false, false>(L, stream));
  return bf16 ? (tree ? launch_t<64, true, true>(L, stream) : launch_t<64, true, false>(L, stream))
              : (tree ? launch_t<64, false, true>(L, stream) : launch_t<64, false, false>(L, stream));
}

}  // namespace fa
