// Attention over packed sequences of different lengths with grouped K/V heads, for sm_103a:
// whole prompts (K and V packed like Q) and chunks of new tokens over a paged cache.
//
// Per sequence, query head h and K/V head h / G: O = softmax(scale Q K^T + mask) V, computed
// block by block with the running maximum and sum of the tiled forward (fa_prefill.cu).
//
// Tiles. The G heads of a group read the same K/V, so they share its tile loads: a tensor-core
// tile of 128 rows holds TPT = 128 / G tokens times the G heads, which one TMA box of
// (64 elements of d, G heads, TPT tokens) brings in that order. Besides the G-fold smaller K/V
// traffic, a tile of few tokens wastes little of the key block that crosses the causal
// diagonal, and a single token still fills G rows.
//
// Three kernels:
//   var_plan_kernel   one CTA: reads the lengths on the device, lists the work items (two
//                     tiles over the key blocks they see) from most key blocks to fewest, and
//                     splits their key blocks when there are too few items for the SMs.
//   var_fwd_kernel    persistent, one CTA per SM, which takes the list's items in a snake
//                     order. Warps 0-3 and 4-7 are the softmax of tiles A and B (TMEM lane =
//                     row, a whole row per thread), warp 8 loads by TMA, warp 9 issues the
//                     MMAs, warps 10 and 11 store outputs. Tensor-pipe order S_A S_B | PV_A S_A' |
//                     PV_B S_B' | ..., so that one tile's softmax runs while the tensor core
//                     works for the other; with one tile S(0) | S(1) PV(0) | S(2) PV(1) | ...
//   var_merge_kernel  joins the partial results of split items.
//
// Bounds. In the middle of an item a key block takes about 3000 cycles for both tiles, the issue
// and the latencies of the softmax's instructions (2 x 16384 exponentials with their maxima,
// scaling and rounding), against 2600 cycles of MMAs; the special-function units alone are not the
// limit (a third busy in the same softmax of fa_prefill.cu). Around it an item takes about 3000
// more: the last P V, the output, the next item's first scores. 14266 tokens in 8 sequences, 32/8
// heads of 128, bf16, causal: 198 to 209 us from one GPU to another, 1214 to 1280 TFLOP/s (63 to
// 66 % of 1923.5 measured); 4 x 4096 tokens: 1467. Whole tiles leave through ring slots held back for them and a TMA store, because 32 rows per warp
// instruction kept the load/store unit, and with it every other warp's loads, busy for 2000
// cycles (211 -> 203 us). Branches inside the softmax that skip hidden columns cost more than
// they save (199 -> 212 us).
//
// Rows of V behind a sequence's last key belong to the next sequence, or are a page's unused
// slots: their probability is 0, but 0 times an infinity or NaN is not. The MMA warp zeroes
// them in shared memory before the block's P V; the scores of such keys are replaced by -inf.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <climits>
#include <cstdint>

#include "fa_mma.cuh"
#include "fa_plan.h"
#include "fa_ptx.cuh"
#include "fa_varlen.h"
#include "fa_varlen_plan.cuh"

namespace fa {
namespace {

constexpr int kTile = 128;     // rows of a tile (= TMEM lanes)
constexpr int BN = kVarBN;
constexpr float kTau = 8.0f;   // lazy-rescale threshold, log2 units
constexpr uint32_t kSmemLimit = 232448;
constexpr int kThreads = 384;
constexpr int kTmaWarp = 8;
constexpr int kMmaWarp = 9;
constexpr int kStoreWarp = 10;  // and 11: outputs of tiles A and B
// launched at 168 registers per thread: 128 x (200 + 200 + 104) = 384 x 168
constexpr uint32_t kRegsSoftmax = 200;
constexpr uint32_t kRegsProducer = 104;

// Wait that ignores the abort flag (used while winding down).
__device__ __forceinline__ void mbar_wait_quiet(uint32_t bar, uint32_t parity, const WaitCtx& wc) {
  volatile uint32_t zero = 0;
  WaitCtx w2 = wc;
  w2.abort = &zero;
  mbar_wait(bar, parity, w2);
}

// 3-D tiled bulk-tensor store shared -> global of this thread's bulk group; then the group is
// closed and waited for until its reads of shared memory are done.
__device__ __forceinline__ void tma_store_3d(const void* map, uint32_t src, int x, int y, int z) {
  asm volatile(
      "cp.async.bulk.tensor.3d.global.shared::cta.bulk_group [%0, {%2, %3, %4}], [%1];" ::"l"(
          reinterpret_cast<uint64_t>(map)),
      "r"(src), "r"(x), "r"(y), "r"(z)
      : "memory");
}
__device__ __forceinline__ void bulk_commit_and_wait_read() {
  asm volatile("cp.async.bulk.commit_group;" ::: "memory");
  asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
}

// ------------------------------------------------------------------ masks by key position

// Key blocks seen by queries at key positions [lo, hi) of a sequence with sk keys.
__device__ __forceinline__ Range blocks_seen(int lo, int hi, int sk, const PrefillParams& m) {
  PrefillParams f;
  f.mask_mode = m.mask_mode;
  f.window = m.window;
  f.n_global = m.n_global;
  f.Sq = sk;  // positions instead of query indices
  return key_range(lo, hi, BN, sk, f, 0);
}

// The j-th visited block of a unit.
__device__ __forceinline__ int block_at(const VarUnit& u, int j) {
  return j < u.a_end ? j : u.b_start + (j - u.a_end);
}

// Every query at positions [lo, hi] sees every key of the block at n0 (and all are in range).
__device__ __forceinline__ bool block_full(int lo, int hi, int n0, int sk,
                                           const PrefillParams& m) {
  const int n1 = n0 + BN;
  if (n1 > sk) return false;
  switch (m.mask_mode) {
    case FA_MASK_NONE:
      return true;
    case FA_MASK_BAND:
      return static_cast<long long>(hi) - n0 <= m.window &&
             static_cast<long long>(n1 - 1) - lo <= m.window;
    case FA_MASK_PREFIX_LM:
      return n1 <= m.n_global || n1 - 1 <= lo;
    case FA_MASK_CAUSAL:
      return n1 - 1 <= lo;
    default:
      return n1 - 1 <= lo && (n1 <= m.n_global || hi - max(n0, m.n_global) < m.window);
  }
}

// Scores of the hidden keys of one row to -inf: per 32 columns a bit mask of the visible
// ones, c <= lim and (c >= lo or c < gl).
__device__ __forceinline__ void mask_row(uint32_t* s, int n0, int pos, int sk,
                                         const PrefillParams& m) {
  int lim = min(pos, sk - 1) - n0, lo = INT_MIN, gl = INT_MIN;
  if (m.mask_mode == FA_MASK_NONE) {
    lim = sk - 1 - n0;
  } else if (m.mask_mode == FA_MASK_CAUSAL_WINDOW) {
    const long long l0 = static_cast<long long>(pos) - m.window + 1 - n0;
    lo = l0 < INT_MIN ? INT_MIN : static_cast<int>(l0);
    gl = m.n_global - n0;
  } else if (m.mask_mode == FA_MASK_BAND) {
    const long long hi = static_cast<long long>(pos) + m.window;
    lim = static_cast<int>((hi < sk - 1 ? hi : sk - 1) - n0);
    const long long l0 = static_cast<long long>(pos) - m.window - n0;
    lo = l0 < INT_MIN ? INT_MIN : static_cast<int>(l0);
  } else if (m.mask_mode == FA_MASK_PREFIX_LM) {
    lim = min(max(pos, m.n_global - 1), sk - 1) - n0;
  }
  lim = max(lim, -1);
  lo = max(lo, -1);
  gl = max(gl, 0);
#pragma unroll
  for (int k = 0; k < BN / 32; ++k) {
    const int b = lim - 32 * k, a = lo - 32 * k, g = gl - 32 * k;
    const uint32_t upto = b < 0 ? 0u : (b >= 31 ? 0xffffffffu : (2u << b) - 1u);
    const uint32_t from = a <= 0 ? 0xffffffffu : (a >= 32 ? 0u : ~((1u << a) - 1u));
    const uint32_t below = g <= 0 ? 0u : (g >= 32 ? 0xffffffffu : (1u << g) - 1u);
    const uint32_t mk = upto & (from | below);
#pragma unroll
    for (int c = 0; c < 32; ++c)
      if (!((mk >> c) & 1u)) s[32 * k + c] = __float_as_uint(-INFINITY);
  }
}

// ------------------------------------------------------------------ plan

constexpr int kCandidates = 32;   // split sizes tried, one per warp of the plan kernel
constexpr int kSplitBelow = 512;  // units (of one K/V head) above which nothing is split
static_assert(kCandidates * 32 == kPlanThreads, "a warp per candidate");

struct PlanSmem {
  SeqScan<kPlanThreads> scan;
  int bins[kBins + 1];
  // units and the most key blocks of one (used for few units alone), split choice
  int pairs, n_max, slots, groups, split;
  int blocks[kSplitBelow];  // key blocks of the units, while there are few
  int split_of[kCandidates];
  float cost_of[kCandidates];
};

// Calls f(unit) for every token block of every sequence (one unit of all its key blocks).
template <typename F>
__device__ __forceinline__ void for_each_block(const VarParams& p, PlanSmem& s, bool report,
                                               F f) {
  const int tpi = 2 * p.TPT;
  for_each_part(
      s.scan, p.B,
      [&](int b) {
        SeqRows r = rows_of(p.cu_q, b, p.total_q);
        Seq q{r.first, r.n, 0, 0, 0};
        bool bad = r.bad;
        if (p.block_table) {
          const int cap = p.page_size * p.max_pages, sk = p.ctx[b];
          bad = bad || sk < 0 || sk > cap;
          q.sk = sk < 0 ? 0 : min(sk, cap);
        } else {
          r = rows_of(p.cu_k, b, p.total_k);
          bad = bad || r.bad;
          q.k0 = r.first;
          q.sk = r.n;
        }
        if (bad && report) atomicOr(p.m.status, FA_DEV_BAD_PAGE);
        q.parts = (q.sq + tpi - 1) / tpi;
        return q;
      },
      [&](int b, const Seq& q, int i) {
        VarUnit u;
        u.q0 = q.q0 + i * tpi;
        u.nq = min(tpi, q.sq - i * tpi);
        u.sk = q.sk;
        u.k0 = q.k0;
        u.qpos = i * tpi + q.sk - q.sq;
        u.seq = b;
        u.j0 = 0;
        const Range rg = blocks_seen(u.qpos, u.qpos + u.nq, u.sk, p.m);
        u.j1 = range_count(rg);
        u.a_end = rg.a_end;
        u.b_start = rg.b_start;
        u.slot = -1;
        f(u);
      });
}

// The work list. Splitting: an item of n key blocks takes about n + 4 block times (the 4:
// first loads, last P V, epilogue); with splits of at most S blocks the launch takes about
// max(S + 4, ceil(items / SMs) (mean + 4)), and 8 more to join them (a 512-token chunk over
// 8192 cached tokens with 8 K/V heads has 64 items for 152 SMs). The least of a few S wins.
//
// One CTA for a few microseconds, most of them spent fetching its instructions: the passes over
// the units share one copy of the code, and units stay in registers when there are no more of
// them than threads.
enum { kCount, kTry, kRecount, kWrite, kPasses };
__global__ void __launch_bounds__(kPlanThreads) var_plan_kernel(const VarParams p, int sms) {
  __shared__ PlanSmem s;
  const int tid = threadIdx.x;
  for (int i = tid; i <= kBins; i += kPlanThreads) s.bins[i] = 0;
  if (tid == 0) {
    s.pairs = s.n_max = s.slots = s.groups = 0;
    s.split = INT_MAX;
  }
  __syncthreads();
  VarUnit mine;       // the last unit this thread has seen
  bool has = false, one_pass = false;
#pragma unroll 1
  for (int pass = kCount; pass < kPasses; ++pass) {
    const int split = s.split, n_max = s.n_max;
    if (pass == kTry) {
      if (!(p.part && s.pairs * p.Hkv < 2 * sms && s.pairs <= kSplitBelow && n_max >= 8)) continue;
      // warp c: sizes from the largest unit (no split) down to a third of an SM's share
      const int c = tid / 32, lane = tid % 32;
      long long cost = 0;  // of all units: 512 of 2^23 key blocks leave 32 bits
      for (int i = lane; i < s.pairs; i += 32) cost += s.blocks[i];
#pragma unroll
      for (int o = 16; o > 0; o /= 2) cost += __shfl_xor_sync(0xffffffffu, cost, o);
      const float lo = fmaxf(4.f, static_cast<float>(cost) * p.Hkv / (3.f * sms));
      const float f = static_cast<float>(kCandidates - 1 - c) / (kCandidates - 1);
      const int S = c == 0 ? n_max
                           : max(1, min(n_max, static_cast<int>(ceilf(lo * powf(n_max / lo, f)))));
      int units = 0;
      for (int i = lane; i < s.pairs; i += 32) units += max(1, (s.blocks[i] + S - 1) / S);
#pragma unroll
      for (int o = 16; o > 0; o /= 2) units += __shfl_xor_sync(0xffffffffu, units, o);
      if (lane == 0) {
        const int items = units * p.Hkv;
        const bool fits = c == 0 || (items <= kVarMaxSplit && units <= p.max_units);
        const float mean = static_cast<float>(cost) / units;
        s.cost_of[c] = !fits ? INFINITY
                             : fmaxf(S + 4.f, ((items + sms - 1) / sms) * (mean + 4.f)) +
                                   (units > s.pairs ? 8.f : 0.f);
        s.split_of[c] = units > s.pairs ? S : INT_MAX;
      }
      __syncthreads();
      if (tid == 0) {
        int best = 0;
        for (int k = 1; k < kCandidates; ++k)
          if (s.cost_of[k] < s.cost_of[best]) best = k;
        s.split = s.split_of[best];
      }
      __syncthreads();
      continue;
    }
    if (pass == kRecount) {
      if (split == INT_MAX) continue;
      for (int i = tid; i <= kBins; i += kPlanThreads) s.bins[i] = 0;
      __syncthreads();
    }
    if (pass == kWrite) {
      const int units = scan_bins(s.scan, s.bins);
      if (tid == 0) {  // more than fit only when starts overlap, which no packed rows have
        p.hdr->units = max(0, min(units, p.max_units));
        if (units < 0 || units > p.max_units) atomicOr(p.m.status, FA_DEV_BAD_PAGE);
      }
    }
    auto visit = [&](VarUnit u) {
      const int n = u.j1, ns = split == INT_MAX ? 1 : max(1, (n + split - 1) / split);
      if (pass == kCount && p.part) {
        const int i = atomicAdd(&s.pairs, 1);
        if (i < kSplitBelow) s.blocks[i] = n;
        atomicMax(&s.n_max, n);
      }
      if (pass == kWrite && ns > 1) {
        u.slot = atomicAdd(&s.slots, ns);
        p.groups[atomicAdd(&s.groups, 1)] = VarGroup{u.q0, u.nq, u.slot, ns};
      }
      for (int k = 0; k < ns; ++k) {
        u.j0 = static_cast<int>(static_cast<long long>(n) * k / ns);
        u.j1 = static_cast<int>(static_cast<long long>(n) * (k + 1) / ns);
        const int bin = cost_bin(u.j1 - u.j0, p.cost_shift);
        const int at = atomicAdd(&s.bins[pass == kWrite ? bin : bin + 1], 1);
        if (pass == kWrite && at >= 0 && at < p.max_units) p.units[at] = u;
        if (ns > 1) ++u.slot;
      }
    };
    if (one_pass) {
      const bool many = has && split != INT_MAX && mine.j1 > split;
      if (has && !many) visit(mine);
      // split units by the whole warp, one unit after the other, a piece per lane
      for (uint32_t rest = __ballot_sync(0xffffffffu, many); rest; rest &= rest - 1) {
        const int src = __ffs(rest) - 1, lane = tid % 32;
        auto from = [&](int x) { return __shfl_sync(0xffffffffu, x, src); };
        VarUnit u;
        u.q0 = from(mine.q0), u.nq = from(mine.nq), u.sk = from(mine.sk), u.k0 = from(mine.k0);
        u.qpos = from(mine.qpos), u.seq = from(mine.seq);
        u.a_end = from(mine.a_end), u.b_start = from(mine.b_start);
        const int n = from(mine.j1), ns = (n + split - 1) / split;
        int slot = 0;
        if (pass == kWrite && lane == 0) {
          slot = atomicAdd(&s.slots, ns);
          p.groups[atomicAdd(&s.groups, 1)] = VarGroup{u.q0, u.nq, slot, ns};
        }
        slot = __shfl_sync(0xffffffffu, slot, 0);
        for (int k = lane; k < ns; k += 32) {
          u.j0 = static_cast<int>(static_cast<long long>(n) * k / ns);
          u.j1 = static_cast<int>(static_cast<long long>(n) * (k + 1) / ns);
          u.slot = slot + k;
          const int bin = cost_bin(u.j1 - u.j0, p.cost_shift);
          const int at = atomicAdd(&s.bins[pass == kWrite ? bin : bin + 1], 1);
          if (pass == kWrite && at >= 0 && at < p.max_units) p.units[at] = u;
        }
      }
      __syncthreads();
    } else {
      for_each_block(p, s, pass == kCount, [&](const VarUnit& u) {
        mine = u;
        has = true;
        visit(u);
      });
      one_pass = p.B <= kPlanThreads && s.scan.off[p.B] <= kPlanThreads;
    }
  }
  if (tid == 0) p.hdr->groups = s.groups;
}

// ------------------------------------------------------------------ forward

template <int D>
struct Cfg {
  static constexpr int KCH = D / 64;
  static constexpr int Q_BYTES = kTile * D * 2;  // one tile
  static constexpr int TILE_BYTES = BN * D * 2;
  static constexpr int BAR_BYTES = 1024;
  static constexpr int FIT = (int)((kSmemLimit - 1024 - BAR_BYTES - 2 * Q_BYTES) / TILE_BYTES);
  static constexpr int NSLOT = FIT > 8 ? 8 : FIT;
  static constexpr int SMEM = 1024 + 2 * Q_BYTES + NSLOT * TILE_BYTES + BAR_BYTES;
  static constexpr int TMEM_COLS = 512;  // S_A S_B [0, 256), O_A O_B [256, 256 + 2 D)
  static_assert(2 * BN + 2 * D <= 512, "TMEM over budget");
};

struct Bars {
  uint64_t full[8], empty[8];
  uint64_t q_full[2], q_empty[2];
  uint64_t s_full[3], p_full[3];  // tiles A and B; odd blocks of an item with one tile
  uint64_t pv_done[2], o_empty[2];
  uint64_t pv_step;      // every P V of an item with one tile
  uint64_t o_staged[2];  // the tile's output is in shared memory
  uint64_t final_mma;
  uint32_t tmem_base;
  uint32_t abort;
};

// A work item: its unit, K/V head, and tiles (1 when the second has no token).
struct Item {
  VarUnit u;
  int kvh;
  int tiles;
  // The output of tile q leaves through shared memory: a whole tile of final results. (A TMA
  // store writes whole boxes, and what is behind a sequence's last token is not its own.)
  __device__ __forceinline__ bool staged(int q, int TPT) const {
    return u.slot < 0 && u.j1 > u.j0 && u.nq >= (q + 1) * TPT;
  }
};

// The items of this CTA one after the other, in snake order over a list sorted by cost: round r
// covers items r G .. r G + G - 1, backwards on odd rounds. AHEAD: the words of the item to come
// are loaded while the present one is worked on (the softmax warps have no registers for that,
// and have to wait for the item's first scores anyway).
template <bool AHEAD>
struct Items {
  int total, round, t;  // t: the item whose words are in a, b, c; total when there is none
  int4 a, b, c;
  __device__ __forceinline__ void fetch(const VarParams& p) {
    const int G = gridDim.x;
    t = total;
    while (round * G < total) {
      const int x = item_of_round(round++, G, blockIdx.x);
      if (x < total) {
        t = x;
        break;
      }
    }
    if (t < total) {
      const int4* src = reinterpret_cast<const int4*>(p.units + t / p.Hkv);
      a = src[0];
      b = src[1];
      c = src[2];
    }
  }
  __device__ __forceinline__ Items(const VarParams& p, int total) : total(total), round(0) {
    if (AHEAD) fetch(p);
  }
  __device__ __forceinline__ bool next(const VarParams& p, Item& it) {
    if (!AHEAD) fetch(p);
    if (t >= total) return false;
    it.u.q0 = a.x, it.u.nq = a.y, it.u.sk = a.z, it.u.k0 = a.w;
    it.u.qpos = b.x, it.u.seq = b.y, it.u.j0 = b.z, it.u.j1 = b.w;
    it.u.slot = c.x, it.u.a_end = c.y, it.u.b_start = c.z;
    it.kvh = t % p.Hkv;
    it.tiles = it.u.nq > p.TPT ? 2 : 1;
    if (AHEAD) fetch(p);
    return true;
  }
};

// One row of one S tile by one thread: mask, running maximum, lazy rescale of O and l (only
// when the maximum rose by more than kTau; decided per warp), P = 2^(S sl2 - m) rounded to 16
// bits over S, l += the unrounded sum. P of at most 2^8 and l in FP32 keep the rounding of P
// the only one on the way.
// `before_rescale` makes O safe to touch, false on abort.
template <int D, bool BF16, typename PreRescale>
__device__ __forceinline__ bool softmax_row(uint32_t t_lane, uint32_t s_col, uint32_t o_col,
                                            bool full, int n0, int pos, int sk,
                                            const PrefillParams& m, float& m_ref, float& l,
                                            PreRescale before_rescale) {
  uint32_t s[BN];
  tmem_ld64(t_lane + s_col, s);
  tmem_ld64(t_lane + s_col + 64, s + 64);
  tmem_ld_wait<BN>(s);
  if (!full) mask_row(s, n0, pos, sk, m);
  float mx[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    mx[i] = fmaxf(__uint_as_float(s[2 * i]), __uint_as_float(s[2 * i + 1]));
#pragma unroll
  for (int c = 8; c < BN; c += 8)
#pragma unroll
    for (int i = 0; i < 4; ++i)
      mx[i] = max3f(mx[i], __uint_as_float(s[c + 2 * i]), __uint_as_float(s[c + 2 * i + 1]));
  const float m_new = fmaxf(m_ref, max3f(mx[0], mx[1], fmaxf(mx[2], mx[3])) * m.sl2);
  const bool need = m_ref != -INFINITY && m_new > m_ref + kTau;
  if (m_ref == -INFINITY) m_ref = m_new;
  if (__any_sync(0xffffffffu, need)) {
    if (!before_rescale()) return false;
    const float alpha = need ? ex2_approx(m_ref - m_new) : 1.f;
    if (need) {
      l *= alpha;
      m_ref = m_new;
    }
#pragma unroll 1
    for (int c = 0; c < D / 32; ++c) {
      uint32_t ov[32];
      tmem_ld32(t_lane + o_col + c * 32, ov);
      tmem_ld_wait<32>(ov);
#pragma unroll
      for (int e = 0; e < 32; ++e) ov[e] = __float_as_uint(__uint_as_float(ov[e]) * alpha);
      tmem_st32(t_lane + o_col + c * 32, ov);
    }
  }
  const float m_use = m_ref == -INFINITY ? 0.f : m_ref;
  const uint64_t scale2 = f2(m.sl2, m.sl2), neg_m2 = f2(-m_use, -m_use);
  uint64_t acc[4] = {0, 0, 0, 0};
#pragma unroll
  for (int c = 0; c < BN; c += 2) {
    const uint64_t x =
        f2_fma(f2(__uint_as_float(s[c]), __uint_as_float(s[c + 1])), scale2, neg_m2);
    float x0, x1;
    f2_split(x, x0, x1);
    const float p0 = ex2_approx(x0), p1 = ex2_approx(x1);
    acc[(c / 2) & 3] = f2_add(acc[(c / 2) & 3], f2(p0, p1));
    s[c / 2] = BF16 ? cvt_pack_bf16(p0, p1) : cvt_pack_f16(p0, p1);
  }
  float a0, a1;
  f2_split(f2_add(f2_add(acc[0], acc[1]), f2_add(acc[2], acc[3])), a0, a1);
  l += a0 + a1;
  tmem_st32(t_lane + s_col, s);
  tmem_st32(t_lane + s_col + 32, s + 32);
  tmem_st_wait();
  return true;
}

template <int D, bool BF16, bool PAGED>
__global__ void __launch_bounds__(kThreads, 1)
    var_fwd_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                   const __grid_constant__ CUtensorMap tmV, const __grid_constant__ CUtensorMap tmO,
                   const __grid_constant__ VarParams p) {
  using C = Cfg<D>;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* smem = smem_raw + (base - raw);
  const uint32_t sQ = base, sRing = base + 2 * C::Q_BYTES;
  Bars* bars = reinterpret_cast<Bars*>(smem + 2 * C::Q_BYTES + C::NSLOT * C::TILE_BYTES);
  auto B = [&](uint64_t& b) { return smem_u32(&b); };
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;

  if (threadIdx.x == 0) {
    for (int i = 0; i < C::NSLOT; ++i) {
      mbar_init(B(bars->full[i]), 1);
      mbar_init(B(bars->empty[i]), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(B(bars->q_full[i]), 1);
      mbar_init(B(bars->q_empty[i]), 1);
      mbar_init(B(bars->pv_done[i]), 1);
      mbar_init(B(bars->o_empty[i]), 128);
      mbar_init(B(bars->o_staged[i]), 128);
    }
    for (int i = 0; i < 3; ++i) {
      mbar_init(B(bars->s_full[i]), 1);
      mbar_init(B(bars->p_full[i]), 128);
    }
    mbar_init(B(bars->pv_step), 1);
    mbar_init(B(bars->final_mma), 1);
    bars->abort = 0;
    mbar_fence_init();
  }
  if (warp == 0) {
    tmem_alloc(smem_u32(&bars->tmem_base), C::TMEM_COLS);
    tmem_relinquish();
  }
  if (warp == kTmaWarp && lane == 0) {
    tma_prefetch_desc(&tmQ);
    tma_prefetch_desc(&tmK);
    tma_prefetch_desc(&tmV);
    tma_prefetch_desc(&tmO);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = bars->tmem_base;
  const WaitCtx wc{&bars->abort, p.m.status, p.m.timeout_ns};
  const int total = p.hdr->units * p.Hkv;
  // The role branches never rejoin: each ends with the CTA-wide teardown barrier, so no code
  // runs under two register budgets.
  if (warp >= 8) {
    regs_decrease<kRegsProducer>();
    if (warp == kTmaWarp) {
      // -------------------------------------------------------------- TMA producer
      const bool leader = elect_one();
      uint32_t pos = 0, iq[2] = {0, 0};
      uint32_t fills[8] = {0, 0, 0, 0, 0, 0, 0, 0};
      bool ok = true;
      Item it;
      const uint32_t q_bytes = static_cast<uint32_t>(p.TPT * p.G) * D * 2;
      for (Items<true> items(p, total); ok && items.next(p, it);) {
        if (it.u.j1 == it.u.j0) continue;
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          if (q >= it.tiles) break;
          if (iq[q] > 0 && !(ok = mbar_wait(B(bars->q_empty[q]), (iq[q] - 1) & 1, wc))) break;
          if (leader) {
            mbar_arrive_expect_tx(B(bars->q_full[q]), q_bytes);
            for (int c = 0; c < C::KCH; ++c)
              tma_load_3d(sQ + q * C::Q_BYTES + c * (kTile * 128), &tmQ, B(bars->q_full[q]),
                          c * 64, it.kvh * p.G, it.u.q0 + q * p.TPT);
          }
          ++iq[q];
        }
        for (int j = it.u.j0; j < it.u.j1 && ok; ++j) {
          const int n0 = block_at(it.u, j) * BN;
          // paged: lane i loads box i of the block, rows of one page; boxes behind the last
          // key are left out
          int y = 0, z = 0, boxes = 1;
          if constexpr (PAGED) {
            boxes = (min(BN, it.u.sk - n0) + p.box - 1) / p.box;
            if (lane < boxes) {
              const int row = n0 + lane * p.box, lp = row / p.page_size;
              int phys = p.block_table[static_cast<size_t>(it.u.seq) * p.max_pages + lp];
              if (phys < 0 || phys >= p.num_pages) {
                atomicOr(p.m.status, FA_DEV_BAD_PAGE);
                phys = 0;
              }
              y = row - lp * p.page_size;
              z = phys * p.Hkv + it.kvh;
            }
          }
          for (int kv = 0; kv < 2; ++kv) {  // K, then V
            const int slot = pos % C::NSLOT;
            const uint32_t use = pos / C::NSLOT;
            if (!(ok = mbar_wait(B(bars->empty[slot]), (use & 1) ^ 1, wc))) break;
            const uint32_t dst = sRing + slot * C::TILE_BYTES;
            const void* map = kv ? (const void*)&tmV : (const void*)&tmK;
            if constexpr (PAGED) {
              if (leader)
                mbar_arrive_expect_tx(B(bars->full[slot]), boxes * p.box * (C::KCH * 128));
              __syncwarp();
              if (lane < boxes)
                for (int c = 0; c < C::KCH; ++c)
                  tma_load_3d(dst + c * (BN * 128) + lane * p.box * 128, map, B(bars->full[slot]),
                              c * 64, y, z);
              __syncwarp();
            } else if (leader) {
              mbar_arrive_expect_tx(B(bars->full[slot]), C::TILE_BYTES);
              for (int c = 0; c < C::KCH; ++c)
                tma_load_3d(dst + c * (BN * 128), map, B(bars->full[slot]), c * 64, it.kvh,
                            it.u.k0 + n0);
            }
            fills[slot] = use + 1;
            ++pos;
          }
        }
      }
      if (!ok) {  // wind down: every load issued lands before the CTA exits
        for (int s = 0; s < C::NSLOT; ++s)
          if (fills[s] > 0) mbar_wait_quiet(B(bars->full[s]), (fills[s] - 1) & 1, wc);
        for (int q = 0; q < 2; ++q)
          if (iq[q] > 0) mbar_wait_quiet(B(bars->q_full[q]), (iq[q] - 1) & 1, wc);
      }
      __syncwarp();
    } else if (warp == kMmaWarp) {
      // -------------------------------------------------------------- MMA issuer
      const bool leader = elect_one();
      const uint32_t tS[2] = {tmem, tmem + BN};
      const uint32_t tO[2] = {tmem + 2 * BN, tmem + 2 * BN + D};
      uint32_t pos = 0, iq[2] = {0, 0}, tc[3] = {0, 0, 0};
      bool ok = true;
      Item it;
      auto qk = [&](int q, int slot) {
        issue_qk<D, BN, BF16>(tS[q], sQ + q * C::Q_BYTES, sRing + slot * C::TILE_BYTES);
        umma_commit(B(bars->s_full[q]));
      };
      // zero the rows of V behind the last key of the j-th visited block
      auto clean = [&](const VarUnit& u, int j, int vslot) {
        const int live = u.sk - block_at(u, u.j0 + j) * BN;  // rows below sk
        if (live >= BN) return;
        uint8_t* v = smem + 2 * C::Q_BYTES + vslot * C::TILE_BYTES;
        for (int c = 0; c < C::KCH; ++c) {
          uint4* r = reinterpret_cast<uint4*>(v + c * (BN * 128));
          for (int i = live * 8 + lane; i < BN * 8; i += 32) r[i] = make_uint4(0, 0, 0, 0);
        }
        fence_proxy_async_smem();
        __syncwarp();
      };
      Items<true> items(p, total);
      for (bool more = items.next(p, it); ok && more;) {
        const int n = it.u.j1 - it.u.j0, last = it.tiles - 1;
        if (n == 0) {
          more = items.next(p, it);
          continue;
        }
        const bool keep[2] = {it.staged(0, p.TPT), it.staged(1, p.TPT)};
        {
          const int slot = pos % C::NSLOT;
          if (!(ok = mbar_wait(B(bars->full[slot]), (pos / C::NSLOT) & 1, wc))) break;
#pragma unroll
          for (int q = 0; q < 2; ++q) {
            if (q >= it.tiles) break;
            if (!(ok = mbar_wait(B(bars->q_full[q]), iq[q] & 1, wc))) break;
            tc_fence_after();
            if (leader) {
              qk(q, slot);
              if (n == 1) umma_commit(B(bars->q_empty[q]));
            }
          }
          if (!ok) break;
          // the last K slot takes tile A's output and the last V slot tile B's, where they leave
          // through shared memory; the store warps then release them
          if (leader && !(n == 1 && keep[0])) umma_commit(B(bars->empty[slot]));
          ++pos;
        }
        Item coming;  // while the first softmax runs
        more = items.next(p, coming);
        // One tile: its scores alternate between both S buffers, so S(j+1) is made while the
        // softmax works on S(j); with P V in between, a block took the whole chain's latency.
        for (int j = 0; j < n && ok && it.tiles == 1; ++j) {
          const int vslot = pos % C::NSLOT, kslot = (pos + 1) % C::NSLOT;
          const bool odd = j & 1;
          if (j + 1 < n) {  // over P(j-1), whose P V is before it in the pipe
            if (!(ok = mbar_wait(B(bars->full[kslot]), ((pos + 1) / C::NSLOT) & 1, wc))) break;
            tc_fence_after();
            if (leader) {
              issue_qk<D, BN, BF16>(tS[odd ? 0 : 1], sQ, sRing + kslot * C::TILE_BYTES);
              umma_commit(B(bars->s_full[odd ? 0 : 2]));
              if (j + 2 == n) umma_commit(B(bars->q_empty[0]));
              if (!(j + 2 == n && keep[0])) umma_commit(B(bars->empty[kslot]));
            }
          }
          if (!(ok = mbar_wait(B(bars->full[vslot]), (pos / C::NSLOT) & 1, wc))) break;
          clean(it.u, j, vslot);
          if (!(ok = mbar_wait(B(bars->p_full[odd ? 2 : 0]), (odd ? tc[2] : tc[0]) & 1, wc))) break;
          if (odd) ++tc[2]; else ++tc[0];
          if (j == 0 && iq[0] > 0 && !(ok = mbar_wait(B(bars->o_empty[0]), (iq[0] - 1) & 1, wc)))
            break;
          tc_fence_after();
          if (leader) {
            issue_pv<D, BN, BF16>(tO[0], tS[odd ? 1 : 0], sRing + vslot * C::TILE_BYTES, j > 0);
            umma_commit(B(bars->pv_step));
            if (j == n - 1) umma_commit(B(bars->pv_done[0]));
            umma_commit(B(bars->empty[vslot]));
          }
          pos += (j + 1 < n) ? 2 : 1;
        }
        for (int j = 0; j < n && ok && it.tiles == 2; ++j) {
          const int vslot = pos % C::NSLOT, kslot = (pos + 1) % C::NSLOT;
          if (!(ok = mbar_wait(B(bars->full[vslot]), (pos / C::NSLOT) & 1, wc))) break;
          clean(it.u, j, vslot);
          tc_fence_after();
#pragma unroll
          for (int q = 0; q < 2; ++q) {
            if (q >= it.tiles) break;
            if (!(ok = mbar_wait(B(bars->p_full[q]), tc[q] & 1, wc))) break;
            ++tc[q];
            tc_fence_after();
            if (j == 0 && iq[q] > 0) {  // the epilogue of the tile's previous item has read O
              if (!(ok = mbar_wait(B(bars->o_empty[q]), (iq[q] - 1) & 1, wc))) break;
              tc_fence_after();
            }
            if (leader) {
              issue_pv<D, BN, BF16>(tO[q], tS[q], sRing + vslot * C::TILE_BYTES, j > 0);
              if (j == n - 1) umma_commit(B(bars->pv_done[q]));
              if (q == last && !(j == n - 1 && keep[1])) umma_commit(B(bars->empty[vslot]));
            }
            if (j + 1 < n) {  // S(j+1) overwrites P(j) only after PV(j) in the pipe
              if (q == 0) {
                if (!(ok = mbar_wait(B(bars->full[kslot]), ((pos + 1) / C::NSLOT) & 1, wc))) break;
                tc_fence_after();
              }
              if (leader) {
                qk(q, kslot);
                if (j + 2 == n) umma_commit(B(bars->q_empty[q]));
                if (q == last && !(j + 2 == n && keep[0])) umma_commit(B(bars->empty[kslot]));
              }
            }
          }
          pos += (j + 1 < n) ? 2 : 1;
        }
        ++iq[0];
        if (it.tiles > 1) ++iq[1];
        it = coming;
      }
      if (leader) umma_commit(B(bars->final_mma));  // all MMAs done before TMEM is released
      mbar_wait_quiet(B(bars->final_mma), 0, wc);
      __syncwarp();
    } else {
      // -------------------------------------------------------------- output of tile q
      const int q = warp - kStoreWarp;
      const bool leader = elect_one();
      uint32_t pos = 0, done = 0;
      Item it;
      for (Items<false> items(p, total); items.next(p, it);) {
        const int n = it.u.j1 - it.u.j0;
        pos += 2 * n;
        if (!it.staged(q, p.TPT)) continue;
        if (!mbar_wait(B(bars->o_staged[q]), done & 1, wc)) break;
        ++done;
        const int slot = (pos - 2 + q) % C::NSLOT;
        if (leader) {
          for (int c = 0; c < C::KCH; ++c)
            tma_store_3d(&tmO, sRing + slot * C::TILE_BYTES + c * (kTile * 128), c * 64,
                         it.kvh * p.G, it.u.q0 + q * p.TPT);
          bulk_commit_and_wait_read();
          mbar_arrive(B(bars->empty[slot]));
        }
        __syncwarp();
      }
      __syncwarp();
    }
    tc_fence_before();
    __syncthreads();  // teardown: every role is done with TMEM and shared memory
    return;
  }
  regs_increase<kRegsSoftmax>();
  // ---------------------------------------------------------------- softmax, tiles A / B
  const int q = warp / 4;
  const int row = (warp % 4) * 32 + lane;
  const uint32_t t_lane = tmem + (static_cast<uint32_t>((warp % 4) * 32) << 16);
  const uint32_t o_col = 2 * BN + q * D;
  const int tok = row / p.G, head = row - (row / p.G) * p.G;  // of the tile, of the group
  // phases behind: this tile's barriers, those of odd blocks of one-tile items, their P Vs
  uint32_t ii = 0, tc = 0, tc_odd = 0, steps = 0, pos = 0;
  bool ok = true;
  Item it;
  for (Items<false> items(p, total); ok && items.next(p, it);) {
    const int n = it.u.j1 - it.u.j0;
    pos += 2 * n;  // ring position behind this item
    if (q >= it.tiles) continue;
    const int left = it.u.nq - q * p.TPT;  // tokens of this tile and behind it
    const int toks = min(p.TPT, left);
    const bool valid = tok < toks;
    const bool work = (warp % 4) * 32 < toks * p.G;  // a warp without rows only keeps step
    const size_t orow = static_cast<size_t>(it.u.q0 + q * p.TPT + tok) * p.H + it.kvh * p.G + head;
    uint16_t* out = static_cast<uint16_t*>(p.o) +
                    static_cast<int64_t>(it.u.q0 + q * p.TPT + tok) * p.o_token +
                    (it.kvh * p.G + head) * D;
    if (n == 0) {  // nothing visible for any row of the item
      if (valid) {
        for (int c = 0; c < D / 8; ++c) reinterpret_cast<uint4*>(out)[c] = make_uint4(0, 0, 0, 0);
        if (p.lse) p.lse[orow] = -INFINITY;
      }
      continue;
    }
    const int p_lo = it.u.qpos + q * p.TPT, p_hi = p_lo + toks - 1, pos_q = p_lo + tok;
    float m_ref = -INFINITY, l = 0.f;
    for (int j = it.u.j0; j < it.u.j1; ++j) {
      const int n0 = block_at(it.u, j) * BN;
      const bool odd = it.tiles == 1 && ((j - it.u.j0) & 1);
      const int bar = odd ? 2 : q;
      ok = mbar_wait(B(bars->s_full[bar]), (odd ? tc_odd : tc) & 1, wc);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      tc_fence_after();
      // With two tiles S(j) was issued after PV(j-1), so O needs no wait before a rescale; with
      // one it was issued before.
      if (work)
        ok = softmax_row<D, BF16>(
            t_lane, odd || q ? BN : 0, o_col, block_full(p_lo, p_hi, n0, it.u.sk, p.m), n0, pos_q,
            it.u.sk, p.m, m_ref, l, [&] {
              if (it.tiles == 2 || j == it.u.j0) return true;
              const bool done = mbar_wait(B(bars->pv_step), (steps + (j - it.u.j0) - 1) & 1, wc);
              tc_fence_after();
              return __all_sync(0xffffffffu, done) != 0;
            });
      if (!ok) break;
      tc_fence_before();
      mbar_arrive(B(bars->p_full[bar]));
      if (odd) ++tc_odd; else ++tc;
    }
    if (!ok) break;
    if (it.tiles == 1) steps += n;
    ok = mbar_wait(B(bars->pv_done[q]), ii & 1, wc);
    ok = __all_sync(0xffffffffu, ok);
    if (!ok) break;
    tc_fence_after();
    if (it.staged(q, p.TPT)) {
      const float inv_l = l != 0.f ? 1.f / l : 0.f;
      // row `row` of the tile in the 128-byte swizzle of its TMA box: conflict-free stores
      const uint32_t dst = sRing + (pos - 2 + q) % C::NSLOT * C::TILE_BYTES + row * 128;
#pragma unroll 1
      for (int c = 0; c < D / 32; ++c) {
        uint32_t ov[32];
        tmem_ld32(t_lane + o_col + c * 32, ov);
        tmem_ld_wait<32>(ov);
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          const float a = __uint_as_float(ov[2 * e]) * inv_l, b = __uint_as_float(ov[2 * e + 1]) * inv_l;
          ov[e] = BF16 ? cvt_pack_bf16(a, b) : cvt_pack_f16(a, b);
        }
#pragma unroll
        for (int e = 0; e < 4; ++e)
          st_shared_v4(dst + (c / 2) * (kTile * 128) +
                           ((static_cast<uint32_t>((c % 2) * 4 + e) ^ (row & 7)) << 4),
                       ov[4 * e], ov[4 * e + 1], ov[4 * e + 2], ov[4 * e + 3]);
      }
      fence_proxy_async_smem();
      mbar_arrive(B(bars->o_staged[q]));
      if (valid && p.lse)
        p.lse[orow] = lse_of(m_ref, l);
    } else if (it.u.slot < 0) {
      const float inv_l = l != 0.f ? 1.f / l : 0.f;
      const bool wide = ((reinterpret_cast<uintptr_t>(p.o) | (p.o_token * 2)) & 31u) == 0;
#pragma unroll 1
      for (int c = 0; c < D / 32; ++c) {
        uint32_t ov[32], pk[16];
        tmem_ld32(t_lane + o_col + c * 32, ov);
        tmem_ld_wait<32>(ov);
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          const float a = __uint_as_float(ov[2 * e]) * inv_l, b = __uint_as_float(ov[2 * e + 1]) * inv_l;
          pk[e] = BF16 ? cvt_pack_bf16(a, b) : cvt_pack_f16(a, b);
        }
        if (valid) {
          if (wide) {
            st_global_v8(out + c * 32, pk);
            st_global_v8(out + c * 32 + 16, pk + 8);
          } else {
#pragma unroll
            for (int e = 0; e < 4; ++e)
              reinterpret_cast<uint4*>(out + c * 32)[e] =
                  make_uint4(pk[4 * e], pk[4 * e + 1], pk[4 * e + 2], pk[4 * e + 3]);
          }
        }
      }
      if (valid && p.lse)
        p.lse[orow] = lse_of(m_ref, l);
    } else {  // partial result: O unnormalised, m in log2 units, l
      float* slot = p.part + (static_cast<size_t>(it.u.slot) * p.Hkv + it.kvh) *
                                 (static_cast<size_t>(kVarSplitRows) * (D + 2));
      const int r = q * kTile + row;
#pragma unroll 1
      for (int c = 0; c < D / 32; ++c) {
        uint32_t ov[32];
        tmem_ld32(t_lane + o_col + c * 32, ov);
        tmem_ld_wait<32>(ov);
        if (valid) {
          uint4* dst = reinterpret_cast<uint4*>(slot + static_cast<size_t>(r) * D + c * 32);
#pragma unroll
          for (int e = 0; e < 8; ++e)
            dst[e] = make_uint4(ov[4 * e], ov[4 * e + 1], ov[4 * e + 2], ov[4 * e + 3]);
        }
      }
      if (valid) {
        slot[kVarSplitRows * D + r] = m_ref;
        slot[kVarSplitRows * (D + 1) + r] = l;
      }
    }
    tc_fence_before();
    mbar_arrive(B(bars->o_empty[q]));
    ++ii;
  }
  tc_fence_before();
  __syncthreads();  // teardown
  if (warp == 0) {
    tc_fence_after();
    tmem_dealloc(tmem, C::TMEM_COLS);
  }
}

// ------------------------------------------------------------------ joining split items

// One warp per row: M = max m_s, O = sum 2^(m_s - M) O_s / sum 2^(m_s - M) l_s over the
// group's slots in order. Rows without a token are skipped.
constexpr int kMergeThreads = 512;
template <int D, bool BF16>
__global__ void __launch_bounds__(kMergeThreads) var_merge_kernel(const VarParams p) {
  constexpr int E = D / 32;  // elements per lane
  const int lane = threadIdx.x % 32;
  const int warps = gridDim.x * (kMergeThreads / 32), per = p.Hkv * kVarSplitRows;
  const size_t step = static_cast<size_t>(p.Hkv) * kVarSplitRows * (D + 2);
  for (int w = blockIdx.x * (kMergeThreads / 32) + threadIdx.x / 32; w / per < kVarMaxSplit;
       w += warps) {
    const int4 gw = reinterpret_cast<const int4*>(p.groups)[w / per];  // beside the count
    if (w / per >= p.hdr->groups) return;
    const VarGroup g{gw.x, gw.y, gw.z, gw.w};
    const int kvh = (w % per) / kVarSplitRows, r = w % kVarSplitRows;
    const int tok = (r / kTile) * p.TPT + (r % kTile) / p.G;
    if ((r % kTile) / p.G >= p.TPT || tok >= g.nq) continue;
    const float* s0 = p.part + (static_cast<size_t>(g.slot) * p.Hkv + kvh) *
                                   (static_cast<size_t>(kVarSplitRows) * (D + 2));
    const float* row = s0 + static_cast<size_t>(r) * D + lane * E;
    constexpr int N = 12;  // slots in flight
    float o[N][E];
    auto load = [&](int s1) {
#pragma unroll
      for (int i = 0; i < N; ++i)
#pragma unroll
        for (int e = 0; e < E; e += 2) {
          const float2 x = s1 + i < g.n ? *reinterpret_cast<const float2*>(row + (s1 + i) * step + e)
                                        : make_float2(0.f, 0.f);
          o[i][e] = x.x;
          o[i][e + 1] = x.y;
        }
    };
    load(0);  // beside the maxima and sums, one slot per lane
    float M = -INFINITY, L = 0.f;
    for (int s1 = 0; s1 < g.n; s1 += 32) {
      float m = -INFINITY, l = 0.f;
      if (s1 + lane < g.n) {
        m = s0[(s1 + lane) * step + kVarSplitRows * D + r];
        l = s0[(s1 + lane) * step + kVarSplitRows * (D + 1) + r];
      }
      float mx = fmaxf(M, m);
#pragma unroll
      for (int i = 16; i > 0; i /= 2) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, i));
      const float mu = mx == -INFINITY ? 0.f : mx;
      l *= ex2_approx(m - mu);
#pragma unroll
      for (int i = 16; i > 0; i /= 2) l += __shfl_xor_sync(0xffffffffu, l, i);
      L = L * ex2_approx(M - mu) + l;
      M = mx;
    }
    const float mu = M == -INFINITY ? 0.f : M;
    float acc[E];
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] = 0.f;
    for (int s1 = 0;;) {
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const float m = s1 + i < g.n ? s0[(s1 + i) * step + kVarSplitRows * D + r] : -INFINITY;
        const float wt = ex2_approx(m - mu);
#pragma unroll
        for (int e = 0; e < E; ++e) acc[e] = fmaf(wt, o[i][e], acc[e]);
      }
      if ((s1 += N) >= g.n) break;
      load(s1);
    }
    const float inv = L != 0.f ? 1.f / L : 0.f;
    const int h = kvh * p.G + (r % kTile) % p.G;
    uint32_t* out = reinterpret_cast<uint32_t*>(
        static_cast<uint16_t*>(p.o) + static_cast<int64_t>(g.q0 + tok) * p.o_token + h * D);
#pragma unroll
    for (int e = 0; e < E; e += 2)
      out[(lane * E + e) / 2] = BF16 ? cvt_pack_bf16(acc[e] * inv, acc[e + 1] * inv)
                                     : cvt_pack_f16(acc[e] * inv, acc[e + 1] * inv);
    if (lane == 0 && p.lse)
      p.lse[static_cast<size_t>(g.q0 + tok) * p.H + h] = lse_of(M, L);
  }
}

template <int D, bool BF16>
cudaError_t launch_t(const VarLaunch& L, cudaStream_t stream) {
  var_plan_kernel<<<1, kPlanThreads, 0, stream>>>(L.p, L.sms);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  auto* k = L.p.block_table ? var_fwd_kernel<D, BF16, true> : var_fwd_kernel<D, BF16, false>;
  constexpr int smem = Cfg<D>::SMEM;
  e = L.p.block_table ? prepare_kernel<var_fwd_kernel<D, BF16, true>>(smem)
                      : prepare_kernel<var_fwd_kernel<D, BF16, false>>(smem);
  if (e != cudaSuccess) return e;
  const int64_t items = static_cast<int64_t>(L.p.max_units) * L.p.Hkv;
  const int grid = static_cast<int>(items < L.sms ? items : L.sms);
  k<<<grid, kThreads, smem, stream>>>(L.tmQ, L.tmK, L.tmV, L.tmO, L.p);
  if ((e = cudaGetLastError()) != cudaSuccess || !L.p.part) return e;
  var_merge_kernel<D, BF16><<<L.sms * 2, kMergeThreads, 0, stream>>>(L.p);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_varlen(const VarLaunch& L, int D, bool bf16, cudaStream_t stream) {
  if (D == 128) return bf16 ? launch_t<128, true>(L, stream) : launch_t<128, false>(L, stream);
  return bf16 ? launch_t<64, true>(L, stream) : launch_t<64, false>(L, stream);
}

}  // namespace fa
