// Attention of a few new rows over an 8-bit paged cache with grouped heads, for sm_103a: fa_few.cu's
// call (decode steps, a couple of drafted tokens, at most 16 rows of tokens x heads of a group) on half
// the bytes, which leaves half the time for the arithmetic of a key.
//
// Products are turned round: S^T = K Q^T and O^T = V^T P^T, with 16 keys (16 channels) as the 16 rows
// of an m16n8k16 MMA and the call's rows as its 8 columns. A step of 4 or 8 heads per K/V head then
// fills the MMAs that it issues, where the rows as the 16 had half or three quarters of them idle, and
// scores, probabilities and output take half the registers: three CTAs per SM instead of two.
//
// Every product is formed in FP16, whatever the call's type: an element of the cache is exact there,
// and so is a row of q over the power of two that brings its largest magnitude to [2^14, 2^15)
// (elements 2^-29 of it and above; what smaller ones lose is 2^-40 of it). K's powers of two multiply
// the FP32 scores. V's, 2^e_j, go with the probabilities, P'_j = 2^(x_j + e_j - r) of x_j = s_j - m (s in
// log2 units, m the row's running maximum), where every row of queries has its own running integer r, 7 to
// 15 below the largest x_j + e_j of the keys that it sees. So keys that it does not see move nothing, terms
// down to 2^-20 of the row's largest keep FP16's eleven bits (the likeliest key's, a power of two, is exact),
// and below them 2^-31 of the largest is lost. The output gets its 2^r back at the end.
//
// ldmatrix moves pairs of bytes: a lane gets four neighbouring channels of a key of K, and two keys
// times two channels of V (transposed). The products take d in that order, and q and the output
// follow it.
//
// Bound by reading K and V once, 2 (d + 1) bytes per key and K/V head: 32 sequences of 128,000 keys
// in all, 32/8 heads of 128, bf16: 51.2 us, 5.15 TB/s, of which the join is 5 and the first tiles' wait
// about 2 (39.5 us at the measured copy rate); 89 to 93 with the same cache in 16 bits. Up to 16 rows;
// with 17 to 32 the products and their scaling, not the bytes, set the pace (20 rows: 121 us, where
// fa_varlen.cu takes 70), so those go there.
#include <cstdint>

#include "fa_few.cuh"

namespace fa {
namespace {

// What a segment costs beside its tiles (q, the join of the warps, the output), in tiles: CTAs get equal
// runs of units, and the first kSegment of a (sequence, K/V head) pair's have no tile. Dealt by tiles
// alone, CTAs with many short sequences kept the others waiting (SMs were busy 68 % of the time:
// 60.9 us in the case above, 50.5 so).
constexpr int kSegment = 2;
constexpr float kTop = 7.0f;  // log2 of the largest P' when r moves; with kTau it stays within FP16

// NB: blocks of 8 rows. BK: keys of a tile, of which a warp takes a quarter.
template <int D, int NB>
struct Cfg {
  static constexpr int MB = kFew8Blocks;          // blocks of 16 keys of a warp
  static constexpr int BK = NW * 16 * MB;
  static constexpr int ROWS = 8 * NB;
  static constexpr int CTAS = NB == 1 ? 3 : 2;    // per SM
  static constexpr int TILE = BK * D;             // K or V of one tile
  static constexpr int SCALES = 2 * BK;           // and the exponent bytes of both
  static constexpr int OROW = D + 4;              // floats of an output row in shared memory
  static constexpr int COMB = 2 * ROWS * OROW * 4;  // two warps' outputs
  static constexpr int STATES = 2 * ROWS * 2 * 4;   // their (m, l)
  static constexpr int BARS = 256;
  static constexpr int BUDGET = 233472 / CTAS - 1024;  // 1 KB taken per CTA
  static constexpr int FIT = (BUDGET - COMB - STATES - BARS) / (2 * TILE + SCALES);
  static constexpr int NST = FIT > 8 ? 8 : FIT;
  static constexpr int SMEM = NST * (2 * TILE + SCALES) + COMB + STATES + BARS;
  static_assert(NST >= 2, "too few stages");
};

__device__ __forceinline__ void compute_sync() {
  asm volatile("bar.sync 1, %0;" ::"n"(kCompute) : "memory");
}
__device__ __forceinline__ void cvt8(uint32_t x, uint32_t& lo, uint32_t& hi) {
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(lo) : "h"(static_cast<uint16_t>(x)));
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(hi) : "h"(static_cast<uint16_t>(x >> 16)));
}
// An 8 x 8 matrix of 16-bit elements, transposed.
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t d;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(x));
  return d;
}
// 2^(b - 127) of an exponent byte: an infinity for 255, a subnormal for 0.
__device__ __forceinline__ float power8(uint32_t b) { return __uint_as_float(max(b << 23, 0x400000u)); }
// The exponent e of a byte's 2^e, a NaN for 255.
__device__ __forceinline__ float exponent8(uint32_t b) {
  return b == 255 ? __uint_as_float(0x7fffffffu) : static_cast<float>(static_cast<int>(b) - 127);
}
// The largest of the eight lanes of a row (those of the same lane % 4).
__device__ __forceinline__ float max8(float x) {
#pragma unroll
  for (int o = 4; o < 32; o *= 2) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, o));
  return x;
}
__device__ __forceinline__ uint32_t load_u8(uint32_t addr) {
  uint32_t x;
  asm volatile("ld.shared.u8 %0, [%1];" : "=r"(x) : "r"(addr) : "memory");
  return x;
}

template <int D, bool BF16, int NB>
__global__ void __launch_bounds__(kThreads, Cfg<D, NB>::CTAS)
    few8_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                const __grid_constant__ FewParams p) {
  using C = Cfg<D, NB>;
  constexpr int BK = C::BK, MB = C::MB, KPW = 16 * MB, CH = D / 16;
  extern __shared__ __align__(1024) uint8_t smem[];
  const uint32_t base = smem_u32(smem);
  constexpr int kBehind = C::NST * (2 * C::TILE + C::SCALES);
  const uint32_t sScales = base + C::NST * 2 * C::TILE;  // K's, then V's of a stage
  float* comb = reinterpret_cast<float*>(smem + kBehind);
  float* states = reinterpret_cast<float*>(smem + kBehind + C::COMB);
  Bars* bars = reinterpret_cast<Bars*>(smem + kBehind + C::COMB + C::STATES);
  auto B = [&](uint64_t& x) { return smem_u32(&x); };
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");  // the joining kernel may come up
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
  const Totals tot = tile_totals<BK, true, kSegment>(p, bars->sum);
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
      const int tiles = few_seq<BK, true>(p, b, false).tiles;
      const int64_t n = tiles ? static_cast<int64_t>(tiles + kSegment) * p.Hkv : 0;
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
      const FewSeq s = few_seq<BK, true>(p, b, false);
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
  w.s = few_seq<BK, true>(p, w.b, false);
  w.kvh = bars->first[1] / (w.s.tiles + kSegment);
  w.j = bars->first[1] - w.kvh * (w.s.tiles + kSegment);  // first unit of the pair
  w.left = static_cast<int>(end - begin);                 // units
  // the tiles [j0, j0 + cnt) of the run in the present pair
  int j0, cnt, take;
  auto segment = [&] {
    take = min(w.left, w.s.tiles + kSegment - w.j);
    j0 = max(w.j - kSegment, 0);
    cnt = max(w.j + take - kSegment, 0) - j0;
  };
  auto advance = [&] {  // to the next pair
    w.left -= take;
    w.j = 0;
    if (++w.kvh < p.Hkv || w.left <= 0) return;
    w.kvh = 0;
    do {
      w.s = few_seq<BK, true>(p, ++w.b, false);
    } while (w.s.tiles == 0);  // ends: `left` units lie ahead
  };
  const WaitCtx wc{&bars->abort, p.m.status, p.m.timeout_ns};

  if (warp == NW) {
    // -------------------------------------------------------------- TMA
    // lane = (K, V, their exponents; box of the tile)
    const bool leader = elect_one();
    const int per_tile = BK / p.box;
    const int kind = lane / per_tile, bx = lane % per_tile;
    uint32_t pos = 0, fills[8] = {0, 0, 0, 0, 0, 0, 0, 0};
    bool ok = true;
    while (w.left > 0 && ok) {
      segment();
      for (int j = j0; j < j0 + cnt && ok; ++j, ++pos) {
        const int n0 = tile_at(w.s.rg, j) * BK;
        const int boxes = (min(BK, w.s.sk - n0) + p.box - 1) / p.box;
        int y = 0, z = 0;
        if (kind < 4 && bx < boxes) {
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
        if (leader) mbar_arrive_expect_tx(B(bars->full[st]), boxes * p.box * (2 * D + 2));
        __syncwarp();
        if (kind < 2 && bx < boxes)
          tma_load_3d(base + (2 * st + kind) * C::TILE + bx * p.box * D,
                      kind ? (const void*)&tmV : (const void*)&tmK, B(bars->full[st]), 0, y, z);
        else if (kind < 4 && bx < boxes)
          bulk_load(sScales + st * C::SCALES + (kind - 2) * BK + bx * p.box,
                    (kind == 2 ? p.k_scales : p.v_scales) + static_cast<int64_t>(z) * p.page_size + y,
                    p.box, B(bars->full[st]));
        __syncwarp();
        fills[st] = use + 1;
      }
      advance();
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
  // lane = (gq, cq): in scores gq is a key (and gq + 8) and 2 cq, 2 cq + 1 are rows of a block
  const int kw = warp, gq = lane / 4, cq = lane % 4;
  uint32_t pos = 0;
  bool ok = true;
  while (w.left > 0) {
    segment();
    if (cnt == 0) {
      advance();
      continue;
    }
    const int rows = w.s.n * p.G;
    // Q fragments straight from global memory (rows past the chunk are zero): row gq of a block,
    // channels 4 cq .. 4 cq + 3 of every 16
    uint32_t qf[NB][CH][2];
    float qs[NB][2];  // BF16: powers of two of rows 2 cq, 2 cq + 1
    int tok[NB][2];   // their tokens
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      const int r = 8 * b + gq, t = r / p.G;
      const uint16_t* src = static_cast<const uint16_t*>(p.q) +
                            static_cast<int64_t>(w.s.q0 + t) * p.q_token +
                            (w.kvh * p.G + r - t * p.G) * D + 4 * cq;
#pragma unroll
      for (int c = 0; c < CH; ++c) {
        const uint2 x = r < rows ? *reinterpret_cast<const uint2*>(src + 16 * c) : make_uint2(0, 0);
        qf[b][c][0] = x.x;
        qf[b][c][1] = x.y;
      }
      float own = 1.f;
      if constexpr (BF16) {
        uint32_t big = 0;  // the largest magnitude, in the high half
#pragma unroll
        for (int c = 0; c < CH; ++c)
#pragma unroll
          for (int h = 0; h < 2; ++h)
            big = max(big, max(qf[b][c][h] & 0x7fff0000u, (qf[b][c][h] << 16) & 0x7fff0000u));
        big = max(big, __shfl_xor_sync(0xffffffffu, big, 1));
        big = max(big, __shfl_xor_sync(0xffffffffu, big, 2));
        int e = static_cast<int>(big >> 23) - 127 - 14;
        if (big >= 0x7f800000u || big == 0) e = 0;  // an infinity or NaN stays one
        e = max(e, -112);
        own = __uint_as_float(static_cast<uint32_t>(127 + e) << 23);
        const float up = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
#pragma unroll
        for (int c = 0; c < CH; ++c)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const uint32_t x = qf[b][c][h];
            qf[b][c][h] = cvt_pack_f16(__uint_as_float(x << 16) * up,
                                       __uint_as_float(x & 0xffff0000u) * up);
          }
      }
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        qs[b][e] = BF16 ? __shfl_sync(0xffffffffu, own, 4 * (2 * cq + e)) : 1.f;
        tok[b][e] = (8 * b + 2 * cq + e) / p.G;
      }
    }
    // tiles that every row sees whole start at most at full_to, and at least at full_from or at
    // most at full_global
    int full_to = w.s.sk - BK, full_from = 0, full_global = INT_MIN;
    {
      const int first = w.s.qpos, last = w.s.qpos + w.s.n - 1;
      if (p.m.mask_mode == FA_MASK_CAUSAL || p.m.mask_mode == FA_MASK_CAUSAL_WINDOW)
        full_to = min(full_to, first - BK + 1);
      if (p.m.mask_mode == FA_MASK_CAUSAL_WINDOW) {
        full_from = last - p.m.window + 1;
        // behind the global keys; or the global keys reach the window
        if (full_from <= p.m.n_global) full_from = 0;
        full_global = p.m.n_global - BK;
      }
      if (p.m.mask_mode == FA_MASK_BAND) {
        const long long to = static_cast<long long>(first) + p.m.window - BK + 1;
        full_to = static_cast<int>(min(static_cast<long long>(full_to), to));
        full_from = last - p.m.window;
      }
      if (p.m.mask_mode == FA_MASK_PREFIX_LM)
        full_to = min(full_to, max(first - BK + 1, p.m.n_global - BK));
      if (p.m.mask_mode == FA_MASK_TREE) full_to = min(full_to, first - BK);
    }
    float m[NB][2], l[NB][2], r[NB][2], o[NB][CH][4];
#pragma unroll
    for (int b = 0; b < NB; ++b) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        m[b][e] = -INFINITY;
        r[b][e] = -1e6f;  // below any term
        l[b][e] = 0.f;
      }
#pragma unroll
      for (int c = 0; c < CH; ++c)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[b][c][e] = 0.f;
    }
    for (int j = j0; j < j0 + cnt; ++j, ++pos) {
      const int n0 = tile_at(w.s.rg, j) * BK;
      const int st = pos % C::NST;
      // a warp that gives up still meets the others at the joins (its results are void)
      ok = ok && mbar_wait(B(bars->full[st]), (pos / C::NST) & 1, wc);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) continue;
      const uint32_t sK = base + 2 * st * C::TILE, sV = sK + C::TILE;
      const uint32_t sc = sScales + st * C::SCALES + kw * KPW;
      const int live = w.s.sk - n0;
      float s[NB][MB][4];
#pragma unroll
      for (int mb = 0; mb < MB; ++mb) {
        float half[NB][2][4];  // even and odd 16-channel steps: two chains of products
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
          for (int e = 0; e < 4; ++e) half[b][0][e] = half[b][1][e] = 0.f;
#pragma unroll
        for (int c = 0; c < CH; c += 2) {
          const int key = kw * KPW + 16 * mb + (lane / 16) * 8 + lane % 8, ch = c + (lane / 8) % 2;
          uint32_t kf[4], a[4];
          ldsm4(sK + key * D + ((ch ^ (D == 128 ? key & 7 : (key >> 1) & 3)) << 4), kf);
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            cvt8(kf[h], a[0], a[2]);
            cvt8(kf[2 + h], a[1], a[3]);
#pragma unroll
            for (int b = 0; b < NB; ++b)
              mma<false>(half[b][h], a, qf[b][c + h][0], qf[b][c + h][1]);
          }
        }
        // an infinite power (of 255) makes the score NaN: f - f is
        const float f0 = power8(load_u8(sc + 16 * mb + gq)), f1 = power8(load_u8(sc + 16 * mb + gq + 8));
        const float z0 = f0 - f0, z1 = f1 - f1;
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float x = half[b][0][e] + half[b][1][e];
            // (the powers together first: x times q's alone may leave FP32 where the score does not)
            const float f = e < 2 ? f0 : f1;
            s[b][mb][e] = fmaf(x, BF16 ? f * qs[b][e % 2] : f, e < 2 ? z0 : z1);
          }
      }
      // hidden keys to -inf where some row does not see the whole tile
      if (n0 > full_to || (n0 < full_from && n0 > full_global)) {
#pragma unroll 1
        for (int b = 0; b < NB; ++b)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            // keys of the tile that the row sees: up to lim, and from lo on or below gl
            const int tk = (8 * b + 2 * cq + i) / p.G;
            const long long at = static_cast<long long>(w.s.qpos) + tk - n0;
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
            if (p.m.mask_mode == FA_MASK_TREE) {
              hi = BK;
              if (tk < w.s.n)
                seen = tree_bits(p.tree + static_cast<size_t>(w.s.q0 + tk) * p.tree_words,
                                 p.tree_words, n0 + kw * KPW - w.s.qpos);
            }
            const int lim =
                min(static_cast<int>(max(-1ll, min(hi, static_cast<long long>(BK)))), last);
            const int lo = static_cast<int>(max(-1ll, min(from, static_cast<long long>(BK))));
#pragma unroll
            for (int mb = 0; mb < MB; ++mb)
#pragma unroll
              for (int t = 0; t < 2; ++t) {
                const int own = 16 * mb + 8 * t + gq, key = kw * KPW + own;
                const bool sees = key <= lim && (key >= lo || key < gl) && ((seen >> own) & 1);
#pragma unroll
                for (int bb = 0; bb < NB; ++bb)
                  if (bb == b && !sees) s[bb][mb][2 * t + i] = -INFINITY;
              }
          }
      }
      // V's exponents (of any key behind the last: its probability is 0)
      float ve[MB][2];
#pragma unroll
      for (int mb = 0; mb < MB; ++mb)
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          const int own = 16 * mb + 8 * t + gq;
          const float e = exponent8(load_u8(sc + BK + own));
          ve[mb][t] = kw * KPW + own < live ? e : 0.f;
        }
      // m moves when some lane finds a score 2^kTau above it (a row's keys are spread over eight lanes); r
      // goes down by the whole part, so that the output's own unit, 2^(m + r), goes up by the rest alone
      float mx[NB][2];
      bool need = false;
#pragma unroll
      for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          mx[b][i] = -INFINITY;
#pragma unroll
          for (int mb = 0; mb < MB; ++mb) mx[b][i] = max3f(mx[b][i], s[b][mb][i], s[b][mb][2 + i]);
          mx[b][i] *= p.m.sl2;
          need = need || mx[b][i] > m[b][i] + kTau;
        }
      if (__any_sync(0xffffffffu, need)) {
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const float x = max8(mx[b][i]);
            float a = 1.f;
            if (x > m[b][i] + kTau) {
              const float up = x - m[b][i], whole = m[b][i] == -INFINITY ? 0.f : floorf(up);
              a = ex2_approx(whole - up);
              l[b][i] *= ex2_approx(-up);
              r[b][i] -= whole;
              m[b][i] = x;
            }
#pragma unroll
            for (int c = 0; c < CH; ++c) {
              o[b][c][i] *= a;
              o[b][c][2 + i] *= a;
            }
          }
      }
      // the row's sum, and its terms' exponents x + e in the scores' place; r moves as m does
      need = false;
#pragma unroll
      for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const float mu = m[b][i] == -INFINITY ? 0.f : m[b][i];
          mx[b][i] = -INFINITY;
#pragma unroll
          for (int mb = 0; mb < MB; ++mb) {
            const float x = fmaf(s[b][mb][i], p.m.sl2, -mu), y = fmaf(s[b][mb][2 + i], p.m.sl2, -mu);
            l[b][i] += ex2_approx(x) + ex2_approx(y);
            s[b][mb][i] = x + ve[mb][0];
            s[b][mb][2 + i] = y + ve[mb][1];
            mx[b][i] = max3f(mx[b][i], s[b][mb][i], s[b][mb][2 + i]);
          }
          need = need || mx[b][i] > r[b][i] + kTop + kTau;
        }
      if (__any_sync(0xffffffffu, need)) {
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const float y = max8(mx[b][i]), to = ceilf(y) - kTop;
            const bool move = y > r[b][i] + kTop + kTau;
            const float a = move ? ex2_approx(r[b][i] - to) : 1.f;
            if (move) r[b][i] = to;
#pragma unroll
            for (int c = 0; c < CH; ++c) {
              o[b][c][i] *= a;
              o[b][c][2 + i] *= a;
            }
          }
      }
      uint32_t pf[NB][MB][2];  // P'^T: keys 2 cq, 2 cq + 1 (and 8 on) of row gq
#pragma unroll
      for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int mb = 0; mb < MB; ++mb)
#pragma unroll
          for (int t = 0; t < 2; ++t)
            pf[b][mb][t] = transpose8(cvt_pack_f16(ex2_approx(s[b][mb][2 * t] - r[b][0]),
                                                   ex2_approx(s[b][mb][2 * t + 1] - r[b][1])));
      if (live < BK) {  // rows of V behind the last key: 0 times what they hold may not be 0
        constexpr int CPR = D / 16;  // 16-byte chunks of a row
        for (int i = lane; i < KPW * CPR; i += 32) {
          const int key = kw * KPW + i / CPR;
          if (key >= live) st_shared_v4(sV + key * D + (i % CPR) * 16, 0, 0, 0, 0);
        }
        fence_proxy_async_smem();  // before the slot's next load
        __syncwarp();
      }
#pragma unroll
      for (int mb = 0; mb < MB; ++mb) {
        const int key = kw * KPW + 16 * mb + ((lane / 8) % 2) * 8 + lane % 8;
#pragma unroll
        for (int c = 0; c < CH; c += 2) {
          const int ch = c + lane / 16;
          uint32_t vf[4], a[2][4];
          ldsm4_t(sV + key * D + ((ch ^ (D == 128 ? key & 7 : (key >> 1) & 3)) << 4), vf);
#pragma unroll
          for (int i = 0; i < 4; ++i)  // (key, channel) pairs side by side to keys side by side
            cvt8(__byte_perm(vf[i], 0, 0x3120), a[i / 2][2 * (i % 2)], a[i / 2][2 * (i % 2) + 1]);
#pragma unroll
          for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int b = 0; b < NB; ++b) mma<false>(o[b][c + h], a[h], pf[b][mb][0], pf[b][mb][1]);
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(B(bars->empty[st]));
    }
    // the output in its own size (by two factors: 2^r may be below FP32's normal range where the output is
    // not), the sums over the lanes of a row
#pragma unroll
    for (int b = 0; b < NB; ++b) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const float h = floorf(0.5f * r[b][i]), u = ex2_approx(h), v = ex2_approx(r[b][i] - h);
#pragma unroll
        for (int c = 0; c < CH; ++c) {
          o[b][c][i] = o[b][c][i] * u * v;
          o[b][c][2 + i] = o[b][c][2 + i] * u * v;
        }
        l[b][i] += __shfl_xor_sync(0xffffffffu, l[b][i], 4);
        l[b][i] += __shfl_xor_sync(0xffffffffu, l[b][i], 8);
        l[b][i] += __shfl_xor_sync(0xffffffffu, l[b][i], 16);
      }
    }
    // join the key groups: the upper half hands its state to the lower, until one is left
#pragma unroll
    for (int half = NW / 2; half >= 1; half /= 2) {
      if (kw >= half && kw < 2 * half) {
        float* dst = comb + (kw - half) * C::ROWS * C::OROW;
        float* sd = states + (kw - half) * 2 * C::ROWS;
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const int r = 8 * b + 2 * cq + i;
#pragma unroll
            for (int c = 0; c < CH; ++c)
              *reinterpret_cast<float2*>(dst + r * C::OROW + 16 * c + 2 * gq) =
                  make_float2(o[b][c][i], o[b][c][2 + i]);
            if (gq == 0) {
              sd[r] = m[b][i];
              sd[C::ROWS + r] = l[b][i];
            }
          }
      }
      compute_sync();
      if (kw < half) {
        const float* src = comb + kw * C::ROWS * C::OROW;
        const float* sd = states + kw * 2 * C::ROWS;
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const int r = 8 * b + 2 * cq + i;
            const float m2 = sd[r], M = fmaxf(m[b][i], m2), mu = M == -INFINITY ? 0.f : M;
            const float x = ex2_approx(m[b][i] - mu), y = ex2_approx(m2 - mu);
            l[b][i] = l[b][i] * x + sd[C::ROWS + r] * y;
            m[b][i] = M;
#pragma unroll
            for (int c = 0; c < CH; ++c) {
              const float2 v = *reinterpret_cast<const float2*>(src + r * C::OROW + 16 * c + 2 * gq);
              o[b][c][i] = o[b][c][i] * x + v.x * y;
              o[b][c][2 + i] = o[b][c][2 + i] * x + v.y * y;
            }
          }
      }
      compute_sync();
    }
    if (kw == 0) {
      const bool whole = j0 == 0 && cnt == w.s.tiles;
      // a piece that starts its pair goes to slot 2x + 1, one that continues it to slot 2x
      const int slot = 2 * blockIdx.x + (j0 == 0 ? 1 : 0);
      const int nslots = 2 * gridDim.x;
      if (!whole && j0 == 0 && threadIdx.x == 0) {
        // the piece that starts a pair says where the rest is: CTAs on to that of its last unit
        const int64_t n = bars->all, own_end = n * (blockIdx.x + 1) / bars->used;
        const int64_t last = own_end - w.left + (w.s.tiles + kSegment - w.j) - 1;
        int x = blockIdx.x + 1;
        while (n * (x + 1) / bars->used <= last) ++x;
        p.heads[blockIdx.x] = FewHead{w.s.q0, rows, w.kvh, x};
      }
#pragma unroll
      for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int r = 8 * b + 2 * cq + i;
          if (r >= rows) continue;
          const int head = w.kvh * p.G + r - tok[b][i] * p.G;
          if (whole) {
            const float inv = l[b][i] != 0.f ? 1.f / l[b][i] : 0.f;
            uint16_t* dst = static_cast<uint16_t*>(p.o) +
                            static_cast<int64_t>(w.s.q0 + tok[b][i]) * p.o_token + head * D + 2 * gq;
#pragma unroll
            for (int c = 0; c < CH; ++c) {
              const float x = o[b][c][i] * inv, y = o[b][c][2 + i] * inv;
              *reinterpret_cast<uint32_t*>(dst + 16 * c) =
                  BF16 ? cvt_pack_bf16(x, y) : cvt_pack_f16(x, y);
            }
            if (gq == 0 && p.lse)
              p.lse[static_cast<size_t>(w.s.q0 + tok[b][i]) * p.H + head] = lse_of(m[b][i], l[b][i]);
          } else {
            float* dst = p.part + (static_cast<size_t>(slot) * C::ROWS + r) * D + 2 * gq;
#pragma unroll
            for (int c = 0; c < CH; ++c)
              *reinterpret_cast<float2*>(dst + 16 * c) = make_float2(o[b][c][i], o[b][c][2 + i]);
            if (gq == 0) {
              float* ml = p.part + static_cast<size_t>(nslots) * C::ROWS * D;
              ml[slot * C::ROWS + r] = m[b][i];
              ml[(nslots + slot) * C::ROWS + r] = l[b][i];
            }
          }
        }
    }
    advance();
  }
}

template <int D, bool BF16, int NB>
cudaError_t launch_t(const FewLaunch& L, cudaStream_t stream) {
  using C = Cfg<D, NB>;
  const int most = NB == 1 ? kFew8MaxCtas : kFewMaxCtas;
  const int grid = C::CTAS * L.sms < most ? C::CTAS * L.sms : most;
  cudaError_t e = prepare_kernel<few8_kernel<D, BF16, NB>>(C::SMEM);
  if (e != cudaSuccess) return e;
  few8_kernel<D, BF16, NB><<<grid, kThreads, C::SMEM, stream>>>(L.tmK, L.tmV, L.p);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  const int rows = L.p.max_q * L.p.G;
  cudaLaunchAttribute early;
  early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  early.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid, rows < 1 ? 1 : rows);
  cfg.blockDim = dim3(kCompute);
  cfg.stream = stream;
  cfg.attrs = &early;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, few_merge_kernel<D, BF16, C::ROWS, true>, L.p);
}
template <int D, bool BF16>
cudaError_t launch_rows(const FewLaunch& L, cudaStream_t stream) {
  return L.p.max_q * L.p.G <= 8 ? launch_t<D, BF16, 1>(L, stream) : launch_t<D, BF16, 2>(L, stream);
}

}  // namespace

cudaError_t launch_few8(const FewLaunch& L, int D, bool bf16, cudaStream_t stream) {
  if (D == 128) return bf16 ? launch_rows<128, true>(L, stream) : launch_rows<128, false>(L, stream);
  return bf16 ? launch_rows<64, true>(L, stream) : launch_rows<64, false>(L, stream);
}

}  // namespace fa
