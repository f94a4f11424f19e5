// Gradients of the packed grouped-head attention (fa_varlen.cu) for sm_103a, recomputing the
// scores from the saved LSE. Per sequence and query head h with its K/V head, D_i = dO_i . O_i:
//   P = exp(scale Q K^T - LSE), dV = P^T dO, dP = dO V^T, dS = P (dP - D),
//   dQ = scale dS K, dK = scale dS^T Q,
// dK and dV summed over the heads that share the K/V head.
//
// That sum decides the layout: a CTA holds one block of 128 keys (TMEM lane = key) and streams
// halves of 64 query rows past it, a row being a (token, head) pair of the group; dK and dV of
// the group then stay in TMEM accumulators, K and V are read once for all its heads, and a short
// sequence or the block on the causal diagonal fills a half with few tokens of many heads.
//
// Kernels:
//   bwd_prep      -LSE log2(e) and -D of every row, whichever sequence it belongs to, and zeros of
//                 the FP32 dQ accumulator (HBM-bound). Beside them one CTA plans: key blocks of all
//                 sequences with the halves that see them, sorted so that the longest start first.
//   bwd_main      per half: S^T = K Q^T and dP^T = V dO^T (tcgen05); P^T and dS^T by the
//                 elementwise warps, P^T in 16 bits over its TMEM columns, dS^T into shared
//                 memory; then dV += P^T dO, dK += dS^T Q, dQ^T = K^T dS^T, the last added into
//                 the accumulator in 16-byte reductions. 576 threads: four elementwise
//                 warpgroups (two per half in flight, 32 columns each), TMA warp, MMA warp.
//   bwd_dq        scales and rounds the accumulator into dq (HBM-bound).
//   bwd_sum       HS > 1 alone: sums the head subsets' dk and dv, in order.
// Bounds. 11343 tokens in 4 sequences, 32/8 heads of 128, bf16, causal: 784 to 817 us from one GPU
// to another, 955 to 995 TFLOP/s over the five products (50 to 52 % of 1923.5 measured); the main
// kernel 657 of them (1187 TFLOP/s, MMAs of N = 64 issued by one thread and the elementwise warps in
// turn), prep 62 and dq 50, both at about 5.5 TB/s of mostly accumulator traffic. 24 short
// sequences, 12/4 heads of 64: 37.5 us, three launches and a CTA's fixed 9 us around 7 halves.
//
// Rows of K, Q and dO behind a sequence's end belong to others: they are zeroed in shared
// memory (0 times an infinity or NaN is not 0), and masked probabilities and dS are set to 0.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <climits>
#include <cstdint>
#include <type_traits>

#include "fa_mma.cuh"
#include "fa_ptx.cuh"
#include "fa_varlen.h"
#include "fa_varlen_plan.cuh"

namespace fa {
namespace {

constexpr int kBT = 128;         // keys per block
constexpr int kHalf = kBwdHalf;  // query rows per half
constexpr int kStages = 4;
constexpr int kThreads = 576;
constexpr int kTmaWarp = 16;
constexpr int kMmaWarp = 17;
constexpr int kEwPerHalf = 256;  // elementwise threads per half (two warpgroups)

// ------------------------------------------------------------------ masks

// The queries (indices in their sequence) that see key position j, as an interval; the
// transpose of the forward's masks with positions = index + delta. Empty when lo > hi.
struct Span {
  int lo, hi;
};
__device__ __forceinline__ Span queries_of(int j, int sq, int delta, const PrefillParams& m) {
  long long lo = 0, hi = sq - 1;
  const long long at = static_cast<long long>(j) - delta;
  switch (m.mask_mode) {
    case FA_MASK_CAUSAL:
      lo = at;
      break;
    case FA_MASK_CAUSAL_WINDOW:
      lo = at;
      if (j >= m.n_global) hi = min(hi, at + m.window - 1);
      break;
    case FA_MASK_BAND:
      lo = at - m.window;
      hi = min(hi, at + m.window);
      break;
    case FA_MASK_PREFIX_LM:
      if (j >= m.n_global) lo = at;
      break;
    default:
      break;
  }
  if (lo < 0) lo = 0;
  if (lo > hi) return Span{1, 0};
  return Span{static_cast<int>(lo), static_cast<int>(hi)};
}

// The queries that see any key of [j0, j0 + n): one interval under every mask.
__device__ __forceinline__ Span queries_of_block(int j0, int n, int sq, int delta,
                                                 const PrefillParams& m) {
  if (n < 1 || sq < 1) return Span{1, 0};
  const int j1 = j0 + n - 1;
  long long lo = 0, hi = sq - 1;
  const long long first = static_cast<long long>(j0) - delta, last = static_cast<long long>(j1) - delta;
  switch (m.mask_mode) {
    case FA_MASK_CAUSAL:
      lo = first;
      break;
    case FA_MASK_CAUSAL_WINDOW:
      lo = first;
      if (j0 >= m.n_global) hi = min(hi, last + m.window - 1);
      break;
    case FA_MASK_BAND:
      lo = first - m.window;
      hi = min(hi, last + m.window);
      break;
    case FA_MASK_PREFIX_LM:
      if (j0 >= m.n_global) lo = first;
      break;
    default:
      break;
  }
  if (lo < 0) lo = 0;
  if (lo > hi) return Span{1, 0};
  return Span{static_cast<int>(lo), static_cast<int>(hi)};
}

// ------------------------------------------------------------------ plan

// The plan is one CTA of bwd_prep: a launch of its own, 1024 threads, put its 4 to 5 us before
// everything else (when it was moved here 24 short sequences went from 43.6 us to 39.1, 11343
// tokens in 4 sequences from 806 to 795). Thousands of tiny sequences lose a little by the fewer threads (4096 of 1 to 8
// tokens, 8 heads on one: 220 -> 229 us; on 12/4 heads they gain, 766 -> 744).
constexpr int kPrepThreads = 256;
struct BwdPlanSmem {
  SeqScan<kPrepThreads> scan;
  int bins[kBins + 1];
  int bad, next;  // cu_q has a bad start; first free slot of such a call
};

// Slots of a call's halves. The halves of sequence b start at slot cu[b] / TPH + b, which needs no
// scan but non-decreasing starts. In a call with a bad start, sequences that are valid by themselves
// may lie in any order and share slots that way; there the plan deals the slots out, and leaves
// each sequence's first one (or -1) in seq_slot.
enum { kCount, kDeal, kWrite };

template <typename F>
__device__ __forceinline__ void for_each_key_block(const VarBwdParams& p, BwdPlanSmem& s,
                                                   int pass, bool dealt, F f) {
  for_each_part(
      s.scan, p.B,
      [&](int b) {
        const SeqRows q = rows_of(p.cu_q, b, p.total_q), k = rows_of(p.cu_k, b, p.total_k);
        if (pass == kCount) {
          if (q.bad || k.bad) atomicOr(p.m.status, FA_DEV_BAD_PAGE);
          if (q.bad) s.bad = 1;
        }
        if (pass == kDeal) {
          const int n = (q.n + p.TPH - 1) / p.TPH;
          int at = n > 0 ? atomicAdd(&s.next, n) : -1;
          if (at < 0 || at > p.slots - n) at = -1;  // only where sequences overlap
          p.seq_slot[b] = at;
        }
        // a sequence whose starts make no sense counts as empty on both sides
        const int sq = k.bad ? 0 : q.n, sk = q.bad ? 0 : k.n;
        return Seq{q.first, sq, k.first, sk, (sk + kBT - 1) / kBT};
      },
      [&](int b, const Seq& q, int i) {
        VarBwdUnit u;
        u.j0 = i * kBT;
        u.k0 = q.k0 + u.j0;
        u.nk = min(kBT, q.sk - u.j0);
        u.q0 = q.q0;
        u.sq = q.sq;
        u.delta = q.sk - q.sq;
        const Span see = queries_of_block(u.j0, u.nk, u.sq, u.delta, p.m);
        u.h0 = see.lo <= see.hi ? see.lo / p.TPH : 0;
        u.n = see.lo <= see.hi ? see.hi / p.TPH - u.h0 + 1 : 0;
        u.slot0 = dealt ? p.seq_slot[b] : q.q0 / p.TPH + b;
        if (u.slot0 < 0) u.h0 = u.n = u.slot0 = 0;
        f(u);
      });
}

__device__ __noinline__ void bwd_plan(const VarBwdParams& p, BwdPlanSmem& s) {
  for (int i = threadIdx.x; i <= kBins; i += kPrepThreads) s.bins[i] = 0;
  if (threadIdx.x == 0) s.bad = s.next = 0;
  __syncthreads();
  // passes that share one copy of the code: counting, counting again while dealing slots (after a
  // bad start), writing; units stay in registers when there are no more of them than threads
  VarBwdUnit mine;
  bool has = false, one_pass = false, dealt = false;
#pragma unroll 1
  for (int pass = kCount; pass <= kWrite; ++pass) {
    if (pass == kDeal) {
      if (!s.bad) continue;
      dealt = true;
      one_pass = false;
      for (int i = threadIdx.x; i <= kBins; i += kPrepThreads) s.bins[i] = 0;
      __syncthreads();
    }
    if (pass == kWrite) {
      const int units = scan_bins(s.scan, s.bins);
      if (threadIdx.x == 0) {  // more than fit only when starts overlap, which no packed rows have
        p.n_units[0] = max(0, min(units, p.max_units));
        p.n_units[1] = dealt;
        if (units < 0 || units > p.max_units) atomicOr(p.m.status, FA_DEV_BAD_PAGE);
      }
    }
    auto visit = [&](const VarBwdUnit& u) {
      const int bin = cost_bin(u.n, p.cost_shift);
      const int at = atomicAdd(&s.bins[pass == kWrite ? bin : bin + 1], 1);
      if (pass == kWrite && at >= 0 && at < p.max_units) p.units[at] = u;
    };
    if (one_pass) {
      if (has) visit(mine);
    } else {
      for_each_key_block(p, s, pass, dealt, [&](const VarBwdUnit& u) {
        mine = u;
        has = true;
        visit(u);
      });
      one_pass = !dealt && p.B <= kPrepThreads && s.scan.off[p.B] <= kPrepThreads;
    }
  }
}

// ------------------------------------------------------------------ passes over half slots

// The tokens of half slot s: first row and number (0: no half lives there).
struct HalfRows {
  int t0, n;
};
// Found by one warp where no start is bad: 32 sequences probed at a time narrow the range 32-fold
// per load.
__device__ __forceinline__ HalfRows half_rows_sorted(const VarBwdParams& p, int s) {
  const int lane = threadIdx.x % 32;
  int lo = 0, n = p.B;  // the last sequence whose slots start at or before s is in [lo, lo + n)
  while (n > 1) {
    const int step = (n + 31) / 32, at = lo + lane * step;
    const bool in = lane * step < n && p.cu_q[at] / p.TPH + at <= s;
    const uint32_t hit = __ballot_sync(0xffffffffu, in);
    const int last = hit ? 31 - __clz(hit) : 0;
    n = min(step, n - last * step);
    lo += last * step;
  }
  const SeqRows r = rows_of(p.cu_q, lo, p.total_q);
  const int at = (s - (r.first / p.TPH + lo)) * p.TPH;
  if (r.bad || at < 0 || at >= r.n) return HalfRows{0, 0};
  return HalfRows{r.first + at, min(p.TPH, r.n - at)};
}
// The same after the plan has run: where slots were dealt out, every sequence is asked.
__device__ __forceinline__ HalfRows half_rows(const VarBwdParams& p, int s) {
  const int dealt = p.n_units[1];  // on its way during the search
  const HalfRows sorted = half_rows_sorted(p, s);
  if (!dealt) return sorted;
  for (int b0 = 0; b0 < p.B; b0 += 32) {
    const int b = b0 + static_cast<int>(threadIdx.x % 32);
    SeqRows r{0, 0, true};
    int i = -1;  // which half of the sequence
    if (b < p.B) {
      r = rows_of(p.cu_q, b, p.total_q);
      if (p.seq_slot[b] >= 0) i = s - p.seq_slot[b];
    }
    const bool hit = i >= 0 && i < (r.n + p.TPH - 1) / p.TPH;
    const uint32_t who = __ballot_sync(0xffffffffu, hit);
    if (who) {
      const int src = __ffs(who) - 1, at = i * p.TPH;
      return HalfRows{__shfl_sync(0xffffffffu, r.first + at, src),
                      __shfl_sync(0xffffffffu, min(p.TPH, r.n - at), src)};
    }
  }
  return HalfRows{0, 0};
}

template <bool BF16>
__device__ __forceinline__ float dot8(const uint4& a, const uint4& b) {
  const uint32_t* ap = reinterpret_cast<const uint32_t*>(&a);
  const uint32_t* bp = reinterpret_cast<const uint32_t*>(&b);
  float acc = 0.f;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    float2 x, y;
    if (BF16) {
      x = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(ap + e));
      y = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(bp + e));
    } else {
      x = __half22float2(*reinterpret_cast<const __half2*>(ap + e));
      y = __half22float2(*reinterpret_cast<const __half2*>(bp + e));
    }
    acc += x.x * y.x + x.y * y.y;
  }
  return acc;
}

// Statistics of rows 64 s .. 64 s + 63 of head subset hh (row: token, head), tokens [t0, t1) alone.
template <int D, bool BF16>
__device__ __forceinline__ void prep_rows(const VarBwdParams& p, int hh, int s, int t0, int t1) {
  constexpr int LPR = D / 8;               // lanes per row, 16 bytes each
  constexpr int RPP = kPrepThreads / LPR;  // rows per pass
  const int64_t row0 = static_cast<int64_t>(s) * kHalf;
  if (row0 >= static_cast<int64_t>(t1) * p.GS) return;
  float* nl = p.stats + static_cast<size_t>(hh) * p.total_q * p.GS;
  float* nd = nl + static_cast<size_t>(p.total_q) * p.H;
  const int c = threadIdx.x % LPR;
#pragma unroll
  for (int r0 = 0; r0 < kHalf; r0 += RPP) {
    // total_q H fits 32 bits, and so does what is at most 63 rows behind it, without a sign
    const uint32_t row = static_cast<uint32_t>(row0) + r0 + threadIdx.x / LPR;
    const uint32_t tok = row / static_cast<uint32_t>(p.GS);
    const bool live = tok >= static_cast<uint32_t>(t0) && tok < static_cast<uint32_t>(t1);
    const int64_t t = tok;
    const int h = hh * p.GS + static_cast<int>(row - tok * p.GS);
    float d = 0.f;
    if (live)
      d = dot8<BF16>(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p.o) +
                                                    t * p.o_token + h * D)[c],
                     reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p.dout) +
                                                    t * p.dout_token + h * D)[c]);
#pragma unroll
    for (int off = LPR / 2; off > 0; off /= 2) d += __shfl_xor_sync(0xffffffffu, d, off);
    if (c == 0 && live) {
      nl[row] = -p.lse[t * p.H + h] * 1.4426950408889634f;
      nd[row] = -d;
    }
  }
}

template <int D>
__device__ __forceinline__ void zero_slot(const VarBwdParams& p, int hh, int s) {
  float4* acc = reinterpret_cast<float4*>(
      p.dqacc + (static_cast<size_t>(hh) * p.slots + s) * (kHalf * D));
  for (int i = threadIdx.x; i < kHalf * D / 4; i += kPrepThreads)
    acc[i] = make_float4(0.f, 0.f, 0.f, 0.f);
}

// What the other CTAs may have left out after a bad start, by the plan's CTA: rows from token
// t_end on, and slots that they did not take for a half.
template <int D, bool BF16>
__device__ __noinline__ void prep_rest(const VarBwdParams& p, int t_end) {
  for (int s = 0; s < p.slots; ++s)
    for (int hh = 0; hh < p.Hkv * p.HS; ++hh) {
      if (s >= static_cast<int64_t>(t_end) * p.GS / kHalf)
        prep_rows<D, BF16>(p, hh, s, t_end, p.total_q);
      zero_slot<D>(p, hh, s);
    }
}

template <int D, bool BF16>
__global__ void __launch_bounds__(kPrepThreads, 6)
    bwd_prep_kernel(const __grid_constant__ VarBwdParams p) {
  __shared__ BwdPlanSmem plan;
  __shared__ bool used;
  // rows behind the last start are nobody's, unless a start is bad
  const int t_end = max(0, min(p.cu_q[p.B], p.total_q));
  if (blockIdx.x == 0) {  // the plan, beside the other CTAs' work
    if (blockIdx.y == 0) {
      bwd_plan(p, plan);
      if (plan.bad && p.total_q > 0) prep_rest<D, BF16>(p, t_end);
    }
    return;
  }
  const int s = blockIdx.x - 1;
  if (s > t_end / p.TPH + p.B) return;  // and so are slots behind the last one
  if (threadIdx.x < 32) {
    const HalfRows f = half_rows_sorted(p, s);
    if (threadIdx.x == 0) used = f.n > 0;
  }
  prep_rows<D, BF16>(p, blockIdx.y, s, 0, t_end);
  __syncthreads();
  if (used) zero_slot<D>(p, blockIdx.y, s);
}

// dq of one half: the accumulator's [16 groups][D][4] transposed through shared memory.
template <int D, bool BF16>
__global__ void __launch_bounds__(256) bwd_dq_kernel(const VarBwdParams p) {
  __shared__ __align__(16) float tile[kHalf][D + 4];
  __shared__ HalfRows sh;
  const int hh = blockIdx.y;
  const int kvh = hh / p.HS, h0 = kvh * p.G + (hh % p.HS) * p.GS;
  if (threadIdx.x < 32) {
    const HalfRows f = half_rows(p, blockIdx.x);
    if (threadIdx.x == 0) sh = f;
  }
  __syncthreads();
  const HalfRows r = sh;
  if (r.n == 0) return;
  const size_t slot = static_cast<size_t>(hh) * p.slots + blockIdx.x;
  const float4* acc = reinterpret_cast<const float4*>(p.dqacc + slot * kHalf * D);
  const int rows = r.n * p.GS, groups = (rows + 3) / 4;
  for (int i = threadIdx.x; i < groups * D; i += 256) {
    const float4 v = acc[i];
    const int g = i / D, e = i % D;
    tile[4 * g][e] = v.x;
    tile[4 * g + 1][e] = v.y;
    tile[4 * g + 2][e] = v.z;
    tile[4 * g + 3][e] = v.w;
  }
  __syncthreads();
  for (int i = threadIdx.x; i < rows * (D / 8); i += 256) {
    const int row = i / (D / 8), c = i % (D / 8), tok = row / p.GS;
    const float* src = &tile[row][8 * c];
    uint32_t pk[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float a = src[2 * e] * p.scale, b = src[2 * e + 1] * p.scale;
      pk[e] = BF16 ? cvt_pack_bf16(a, b) : cvt_pack_f16(a, b);
    }
    uint16_t* dst = static_cast<uint16_t*>(p.dq) + (r.t0 + tok) * p.dq_token +
                    (h0 + row - tok * p.GS) * D;
    reinterpret_cast<uint4*>(dst)[c] = make_uint4(pk[0], pk[1], pk[2], pk[3]);
  }
}

// dk and dv of a quarter of the keys of one unit and K/V head: the head subsets' partials summed
// in order.
template <int D, bool BF16>
__global__ void __launch_bounds__(256) bwd_sum_kernel(const VarBwdParams p) {
  const int unit = blockIdx.x / 4, r0 = (blockIdx.x % 4) * (kBT / 4);
  if (unit >= p.n_units[0]) return;
  const int k0 = p.units[unit].k0, nk = p.units[unit].nk;
  const int kvh = blockIdx.y;
  const size_t plane = static_cast<size_t>(p.total_k) * p.Hkv * D;
  constexpr int CH = D / 4;  // 16-byte chunks of a row
#pragma unroll
  for (int i = threadIdx.x; i < 2 * (kBT / 4) * CH; i += 256) {
    const int which = i / ((kBT / 4) * CH), row = r0 + (i / CH) % (kBT / 4), c = i % CH;
    if (row >= nk) continue;
    const float* src = p.part + which * plane + (static_cast<size_t>(k0 + row) * p.Hkv + kvh) * D + 4 * c;
    float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
    for (int s = 0; s < p.HS; ++s) {
      const float4 v = __ldcs(reinterpret_cast<const float4*>(src + 2 * plane * s));
      a.x += v.x, a.y += v.y, a.z += v.z, a.w += v.w;
    }
    const float mul = which ? 1.f : p.scale;
    uint2 o;
    o.x = BF16 ? cvt_pack_bf16(a.x * mul, a.y * mul) : cvt_pack_f16(a.x * mul, a.y * mul);
    o.y = BF16 ? cvt_pack_bf16(a.z * mul, a.w * mul) : cvt_pack_f16(a.z * mul, a.w * mul);
    uint16_t* out = static_cast<uint16_t*>(which ? p.dv : p.dk) +
                    static_cast<int64_t>(k0 + row) * (which ? p.dv_token : p.dk_token) + kvh * D;
    reinterpret_cast<uint2*>(out)[c] = o;
  }
}

// ------------------------------------------------------------------ main kernel

template <int D>
struct Cfg {
  static constexpr int TILE = kBT * D * 2;     // K or V block
  static constexpr int HTILE = kHalf * D * 2;  // Q or dO half
  static constexpr int DS = kBT * kHalf * 2;   // dS^T of one half
  static constexpr int STATS = 2 * kHalf * 4;  // per stage
  static constexpr int BODY = 2 * TILE + kStages * 2 * HTILE + 2 * DS + kStages * STATS + 256;
  static constexpr int WANT = BODY + 1023;  // room to align the base to 1024 bytes
  static constexpr int SMEM = WANT < 232448 ? WANT : 232448;
  static_assert(BODY + 768 <= SMEM, "shared memory over budget");
  // over half the SM's shared memory: one CTA, which takes all 512 TMEM columns, per SM
  static_assert(BODY > 116 * 1024, "two CTAs would share an SM");
};

struct Bars {
  uint64_t res_full;           // K and V landed
  uint64_t st_full[kStages];   // streamed half landed, statistics written
  uint64_t st_empty[kStages];  // MMAs done with the stage
  uint64_t s_full[2];          // S^T and dP^T of the half in TMEM
  uint64_t p_full[2];          // P^T (TMEM) and dS^T (shared memory) written
  uint64_t dq_full[2];         // dQ^T in TMEM (over the dP^T columns)
  uint64_t dq_read[2];         // the elementwise warps have read dQ^T
  uint64_t acc_full;           // every MMA of the CTA complete
  uint32_t tmem_base;
  uint32_t abort;
};
static_assert(sizeof(Bars) <= 256, "barrier block over its reserve");

__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}

__device__ __forceinline__ void tmem_st8(uint32_t taddr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
      : "memory");
}

// Half i of the stream lives in stage i % kStages.
__device__ __forceinline__ int stage_of(int i) { return i % kStages; }
__device__ __forceinline__ uint32_t stage_parity(int i) { return (i / kStages) & 1; }

__device__ __forceinline__ void wait_quiet(uint32_t bar, uint32_t parity, const WaitCtx& wc) {
  volatile uint32_t zero = 0;
  WaitCtx w2 = wc;
  w2.abort = &zero;
  mbar_wait(bar, parity, w2);
}

// X = A B^T: A a resident 128-row tile (64-element regions of d 16 KB apart), B a streamed
// 64-row half (regions 8 KB apart), both K-major; M = 128, N = 64.
template <int D, bool BF16>
__device__ __forceinline__ void issue_s(uint32_t d_tmem, uint32_t a_smem, uint32_t b_half) {
  constexpr uint32_t id = idesc_f16(BF16, kBT, kHalf, false);
  const uint64_t a0 = smem_desc_sw128(a_smem, 16, 1024), b0 = smem_desc_sw128(b_half, 16, 1024);
#pragma unroll
  for (int kk = 0; kk < D / 16; ++kk)
    umma_ss(d_tmem, a0 + static_cast<uint64_t>((kk / 4) * (kBT * 128 / 16) + (kk % 4) * 2),
            b0 + static_cast<uint64_t>((kk / 4) * (kHalf * 128 / 16) + (kk % 4) * 2), id,
            kk > 0 ? 1u : 0u);
}

// dV (+)= P^T dO: A = P^T in TMEM (rows 0-31 of the half in columns [a, a + 16), 32-63 in
// [a + 32, a + 48)), B = the dO half MN-major.
template <int D, bool BF16>
__device__ __forceinline__ void issue_dv(uint32_t y_tmem, uint32_t a_tmem, uint32_t b_half,
                                         bool acc) {
  constexpr uint32_t id = idesc_f16(BF16, kBT, D, true);
  const uint64_t b0 = smem_desc_sw128(b_half, kHalf * 128, 1024);
#pragma unroll
  for (int kk = 0; kk < kHalf / 16; ++kk)
    umma_ts(y_tmem, a_tmem + (kk / 2) * 32 + (kk % 2) * 8, b0 + static_cast<uint64_t>(kk * 128),
            id, (acc || kk > 0) ? 1u : 0u);
}

// dK (+)= dS^T Q: A = dS^T in shared memory (128 keys x 64 rows, K-major), B = the Q half.
template <int D, bool BF16>
__device__ __forceinline__ void issue_dk(uint32_t y_tmem, uint32_t ds, uint32_t b_half, bool acc) {
  constexpr uint32_t id = idesc_f16(BF16, kBT, D, true);
  const uint64_t a0 = smem_desc_sw128(ds, 16, 1024);
  const uint64_t b0 = smem_desc_sw128(b_half, kHalf * 128, 1024);
#pragma unroll
  for (int kk = 0; kk < kHalf / 16; ++kk)
    umma_ss(y_tmem, a0 + static_cast<uint64_t>(kk * 2), b0 + static_cast<uint64_t>(kk * 128), id,
            (acc || kk > 0) ? 1u : 0u);
}

// dQ^T = K^T dS^T (M = D, N = 64, K = 128 keys), both MN-major. With D = 64 the accumulator
// takes the M = 64 layout: row r in TMEM lane 32 (r / 16) + r % 16.
template <int D, bool BF16>
__device__ __forceinline__ void issue_dq(uint32_t y_tmem, uint32_t k_smem, uint32_t ds) {
  constexpr uint32_t id = idesc_f16(BF16, D, kHalf, true, true);
  const uint64_t a0 = smem_desc_sw128(k_smem, kBT * 128, 1024);
  const uint64_t b0 = smem_desc_sw128(ds, kBT * 128, 1024);
#pragma unroll
  for (int kk = 0; kk < kBT / 16; ++kk)
    umma_ss(y_tmem, a0 + static_cast<uint64_t>(kk * 128), b0 + static_cast<uint64_t>(kk * 128), id,
            kk > 0 ? 1u : 0u);
}

// Zero rows [r0, rows) of a tile of 128-byte rows (one region of `rows` rows per 64 elements).
template <int D>
__device__ __forceinline__ void zero_rows(uint8_t* tile, int rows, int r0, int lane, int lanes) {
#pragma unroll
  for (int c = 0; c < D / 64; ++c) {
    uint4* r = reinterpret_cast<uint4*>(tile + c * rows * 128);
    for (int i = r0 * 8 + lane; i < rows * 8; i += lanes) r[i] = make_uint4(0, 0, 0, 0);
  }
}

// TMEM: S^T [0,128) (P^T over the first 16 of every 32 columns), dP^T [128,256) (dQ^T of half u
// over [128 + 64 u, 192 + 64 u) once dP^T has been read), dV [256, 256 + D), dK after it.
template <int D, bool BF16>
__global__ void __launch_bounds__(kThreads, 1)
    bwd_main_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                    const __grid_constant__ CUtensorMap tmV,
                    const __grid_constant__ CUtensorMap tmdO,
                    const __grid_constant__ VarBwdParams p) {
  using C = Cfg<D>;
  const int per = p.Hkv * p.HS;
  const int unit = blockIdx.x / per, hh = blockIdx.x - unit * per;  // hh = kvh HS + subset
  if (unit >= p.n_units[0]) return;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  if (base - raw + C::BODY > static_cast<uint32_t>(C::SMEM)) {  // uniform over the CTA
    if (threadIdx.x == 0) atomicOr(p.m.status, FA_DEV_SMEM_BASE);
    return;
  }
  uint8_t* smem = smem_raw + (base - raw);
  const uint32_t sK = base, sV = base + C::TILE, sSt = base + 2 * C::TILE;
  auto sQ = [&](int h) { return sSt + 2 * h * C::HTILE; };
  auto sdO = [&](int h) { return sSt + (2 * h + 1) * C::HTILE; };
  const uint32_t sDS = sSt + kStages * 2 * C::HTILE;
  float* stats = reinterpret_cast<float*>(smem + 2 * C::TILE + kStages * 2 * C::HTILE + 2 * C::DS);
  Bars* bars = reinterpret_cast<Bars*>(reinterpret_cast<uint8_t*>(stats) + kStages * C::STATS);
  auto B = [&](uint64_t& x) { return smem_u32(&x); };
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;

  VarBwdUnit u;
  {
    const int4* src = reinterpret_cast<const int4*>(p.units + unit);
    const int4 a = src[0], b = src[1], c = src[2];
    u.k0 = a.x, u.nk = a.y, u.j0 = a.z, u.q0 = a.w;
    u.sq = b.x, u.delta = b.y, u.h0 = b.z, u.n = b.w;
    u.slot0 = c.x;
  }
  const int kvh = hh / p.HS, head0 = kvh * p.G + (hh - kvh * p.HS) * p.GS;
  const int used = p.TPH * p.GS;  // rows of a half that a load writes

  if (threadIdx.x == 0) {
    mbar_init(B(bars->res_full), 1);
    for (int i = 0; i < kStages; ++i) {
      mbar_init(B(bars->st_full[i]), 1);
      mbar_init(B(bars->st_empty[i]), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(B(bars->s_full[i]), 1);
      mbar_init(B(bars->p_full[i]), kEwPerHalf);
      mbar_init(B(bars->dq_full[i]), 1);
      mbar_init(B(bars->dq_read[i]), kEwPerHalf);
    }
    mbar_init(B(bars->acc_full), 1);
    bars->abort = 0;
    mbar_fence_init();
  }
  if (used < kHalf) {  // rows that no load writes: zero once
    for (int h = 0; h < 2 * kStages; ++h)
      zero_rows<D>(smem + 2 * C::TILE + h * C::HTILE, kHalf, used, threadIdx.x, kThreads);
    fence_proxy_async_smem();
  }
  if (warp == 0) {
    tmem_alloc(smem_u32(&bars->tmem_base), 512);
    tmem_relinquish();
  }
  if (warp == kTmaWarp && lane == 0) {
    tma_prefetch_desc(&tmQ);
    tma_prefetch_desc(&tmK);
    tma_prefetch_desc(&tmV);
    tma_prefetch_desc(&tmdO);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = bars->tmem_base;
  const WaitCtx wc{&bars->abort, p.m.status, p.m.timeout_ns};
  const size_t slot0 = static_cast<size_t>(hh) * p.slots + u.slot0 + u.h0;  // of half 0

  if (warp == kTmaWarp) {
    // ------------------------------------------------------------ TMA
    const bool leader = elect_one();
    bool ok = true;
    uint32_t fills[kStages] = {0, 0, 0, 0};
    const uint32_t bytes = 2 * static_cast<uint32_t>(used) * D * 2;
    // statistics of the first half: -LSE log2(e) of its rows by lanes 0-15, -D by lanes 16-31; rows
    // that the half does not have hold others' or anything, and are hidden
    const float* src = p.stats + static_cast<size_t>(hh) * p.total_q * p.GS +
                       static_cast<size_t>(u.q0 + u.h0 * p.TPH) * p.GS + (lane % 16) * 4 +
                       (lane < 16 ? 0 : static_cast<size_t>(p.total_q) * p.H);
    const bool wide = p.GS % 4 == 0;
    if (leader && u.n > 0) {
      mbar_arrive_expect_tx(B(bars->res_full), 2 * C::TILE);
#pragma unroll
      for (int c = 0; c < D / 64; ++c)
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const uint32_t off = c * (kBT * 128) + r * (kHalf * 128);
          tma_load_3d(sK + off, &tmK, B(bars->res_full), c * 64, kvh, u.k0 + r * kHalf);
          tma_load_3d(sV + off, &tmV, B(bars->res_full), c * 64, kvh, u.k0 + r * kHalf);
        }
    }
    for (int i = 0; i < u.n && ok; ++i) {
      const int h = stage_of(i);
      // the half's statistics, loaded before the wait for the stage
      const float4 st = wide ? *reinterpret_cast<const float4*>(src)
                             : make_float4(src[0], src[1], src[2], src[3]);
      src += used;
      if (i >= kStages && !(ok = mbar_wait(B(bars->st_empty[h]), stage_parity(i - kStages), wc)))
        break;
      reinterpret_cast<float4*>(stats + h * 2 * kHalf)[lane] = st;
      __syncwarp();  // the leader's arrive below releases every lane's writes
      if (leader) {
        mbar_arrive_expect_tx(B(bars->st_full[h]), bytes);
        const int t = u.q0 + (u.h0 + i) * p.TPH;
#pragma unroll
        for (int c = 0; c < D / 64; ++c) {
          tma_load_3d(sQ(h) + c * (kHalf * 128), &tmQ, B(bars->st_full[h]), c * 64, head0, t);
          tma_load_3d(sdO(h) + c * (kHalf * 128), &tmdO, B(bars->st_full[h]), c * 64, head0, t);
        }
      }
      fills[h] = i / kStages + 1;
    }
    if (!ok) {  // every load issued lands before the CTA exits
      wait_quiet(B(bars->res_full), 0, wc);
      for (int h = 0; h < kStages; ++h)
        if (fills[h] > 0) wait_quiet(B(bars->st_full[h]), (fills[h] - 1) & 1, wc);
    }
    __syncwarp();
  } else if (warp == kMmaWarp) {
    // ------------------------------------------------------------ MMA
    // Per half i (u = i % 2): wait for P^T / dS^T; dV += P^T dO, dK += dS^T Q, release the
    // stage, dQ^T over the dP^T columns; then S^T of half i + 2 over the columns that dV has
    // just read (MMAs of one thread execute in order) and, once dQ^T has been read, its dP^T.
    const bool leader = elect_one();
    bool ok = u.n == 0 || mbar_wait(B(bars->res_full), 0, wc);
    if (ok && u.n > 0 && u.nk < kBT) {  // rows of K behind the last key
      zero_rows<D>(smem, kBT, u.nk, lane, 32);
      fence_proxy_async_smem();
      __syncwarp();
    }
    auto s_half = [&](int i) {
      const int h = stage_of(i);
      if (!(ok = mbar_wait(B(bars->st_full[h]), stage_parity(i), wc))) return;
      const int live = (u.sq - (u.h0 + i) * p.TPH) * p.GS;  // rows of this sequence
      if (live < used) {
        zero_rows<D>(smem + 2 * C::TILE + 2 * h * C::HTILE, kHalf, live, lane, 32);
        zero_rows<D>(smem + 2 * C::TILE + (2 * h + 1) * C::HTILE, kHalf, live, lane, 32);
        fence_proxy_async_smem();
        __syncwarp();
      }
      tc_fence_after();
      if (leader) issue_s<D, BF16>(tmem + 64 * (i & 1), sK, sQ(h));
    };
    auto dp_half = [&](int i) {
      if (leader) {
        issue_s<D, BF16>(tmem + 128 + 64 * (i & 1), sV, sdO(stage_of(i)));
        umma_commit(B(bars->s_full[i & 1]));
      }
    };
    for (int i = 0; i < 2 && i < u.n && ok; ++i) {
      s_half(i);
      if (ok) dp_half(i);
    }
    for (int i = 0; i < u.n && ok; ++i) {
      const int w = i & 1, t = i >> 1, h = stage_of(i);
      if (!(ok = mbar_wait(B(bars->p_full[w]), t & 1, wc))) break;
      tc_fence_after();
      if (leader) {
        issue_dv<D, BF16>(tmem + 256, tmem + 64 * w, sdO(h), i > 0);
        issue_dk<D, BF16>(tmem + 256 + D, sDS + w * C::DS, sQ(h), i > 0);
        umma_commit(B(bars->st_empty[h]));
        issue_dq<D, BF16>(tmem + 128 + 64 * w, sK, sDS + w * C::DS);
        umma_commit(B(bars->dq_full[w]));
      }
      if (i + 2 < u.n) {
        s_half(i + 2);
        if (!ok || !(ok = mbar_wait(B(bars->dq_read[w]), t & 1, wc))) break;
        tc_fence_after();
        dp_half(i + 2);
      }
    }
    if (leader) umma_commit(B(bars->acc_full));
    wait_quiet(B(bars->acc_full), 0, wc);
    __syncwarp();
  } else {
    // ------------------------------------------------------------ elementwise + epilogue
    const int grp = warp / 4, w = grp / 2, sub = grp % 2;  // half w, columns [32 sub, 32 sub + 32)
    const int row = (warp % 4) * 32 + lane;                // key of the block (= TMEM lane)
    const uint32_t t_lane = tmem + (static_cast<uint32_t>((warp % 4) * 32) << 16);
    const uint32_t c_s = 64 * w + 32 * sub;  // this thread's S^T columns; dP^T 128 further
    const uint32_t ds_row = sDS + w * C::DS + row * 128;  // 16-byte chunk c at c ^ (row % 8)
    const int dcol = D == 128 ? row : (lane < 16 ? (warp % 4) * 16 + lane : -1);
    const Span see =
        row < u.nk ? queries_of(u.j0 + row, u.sq, u.delta, p.m) : Span{1, 0};
    bool ok = true;
    for (int i = w; i < u.n && ok; i += 2) {
      const int t = i >> 1, h = stage_of(i), tok0 = (u.h0 + i) * p.TPH;
      // The stage's statistics: it cannot be refilled before this warpgroup has written the P
      // and dS that the MMAs reading it wait for.
      ok = mbar_wait(B(bars->st_full[h]), stage_parity(i), wc);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      const float4* st4 = reinterpret_cast<const float4*>(stats + h * 2 * kHalf + 32 * sub);
      ok = mbar_wait(B(bars->s_full[w]), t & 1, wc);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      tc_fence_after();
      // rows of the half that see this key, [lo, hi], as a bit mask of this thread's columns
      uint32_t mk = 0u;
      {
        const int a = min(max(see.lo - tok0, 0), kHalf) * p.GS - 32 * sub;
        const int b = min(max(see.hi - tok0 + 1, 0), p.TPH) * p.GS - 1 - 32 * sub;
        if (see.lo <= see.hi && a <= b && b >= 0 && a <= 31) {
          const int lo = max(a, 0), hi = min(b, 31);
          mk = (hi >= 31 ? 0xffffffffu : (2u << hi) - 1u) & ~((1u << lo) - 1u);
        }
      }
      const bool all_vis = __all_sync(0xffffffffu, mk == 0xffffffffu);
      auto chunks = [&](auto masked) {
        constexpr bool kMasked = decltype(masked)::value;
#pragma unroll
        for (int c = 0; c < 2; ++c) {  // 16 rows at a time
          uint32_t sv[16], dp[16];
          tmem_ld16(t_lane + c_s + 16 * c, sv);
          tmem_ld16(t_lane + 128 + c_s + 16 * c, dp);
          tmem_ld_wait<16>(sv);
          tmem_ld_tie<16>(dp);
#pragma unroll
          for (int e = 0; e < 16; e += 4) {
            const float4 a = st4[(16 * c + e) / 4];
            const float4 d = st4[kHalf / 4 + (16 * c + e) / 4];
            const uint64_t nl2[2] = {f2(a.x, a.y), f2(a.z, a.w)};
            const uint64_t ndd[2] = {f2(d.x, d.y), f2(d.z, d.w)};
            const uint64_t sl2 = f2(p.m.sl2, p.m.sl2);
            float pv[4], dv[4];
#pragma unroll
            for (int x = 0; x < 4; x += 2) {
              float x0, x1;
              f2_split(f2_fma(f2(__uint_as_float(sv[e + x]), __uint_as_float(sv[e + x + 1])), sl2,
                              nl2[x / 2]), x0, x1);
              const int col = 16 * c + e + x;
              const bool v0 = !kMasked || ((mk >> col) & 1u);
              const bool v1 = !kMasked || ((mk >> (col + 1)) & 1u);
              pv[x] = v0 ? ex2_approx(x0) : 0.f;
              pv[x + 1] = v1 ? ex2_approx(x1) : 0.f;
              const uint64_t dd2 =
                  f2_add(f2(__uint_as_float(dp[e + x]), __uint_as_float(dp[e + x + 1])), ndd[x / 2]);
              f2_split(f2_fma(f2(pv[x], pv[x + 1]), dd2, f2(0.f, 0.f)), dv[x], dv[x + 1]);
              if (kMasked) {  // dP of a hidden pair may be anything
                dv[x] = v0 ? dv[x] : 0.f;
                dv[x + 1] = v1 ? dv[x + 1] : 0.f;
              }
            }
            sv[e / 2] = BF16 ? cvt_pack_bf16(pv[0], pv[1]) : cvt_pack_f16(pv[0], pv[1]);
            sv[e / 2 + 1] = BF16 ? cvt_pack_bf16(pv[2], pv[3]) : cvt_pack_f16(pv[2], pv[3]);
            dp[e / 2] = BF16 ? cvt_pack_bf16(dv[0], dv[1]) : cvt_pack_f16(dv[0], dv[1]);
            dp[e / 2 + 1] = BF16 ? cvt_pack_bf16(dv[2], dv[3]) : cvt_pack_f16(dv[2], dv[3]);
          }
          tmem_st8(t_lane + c_s + 8 * c, sv);  // P^T over columns already read
#pragma unroll
          for (int x = 0; x < 2; ++x)
            st_shared_v4(ds_row + ((static_cast<uint32_t>(4 * sub + 2 * c + x) ^ (row & 7)) << 4),
                         dp[4 * x], dp[4 * x + 1], dp[4 * x + 2], dp[4 * x + 3]);
        }
      };
      if (all_vis)
        chunks(std::false_type{});
      else
        chunks(std::true_type{});
      tmem_st_wait();
      fence_proxy_async_smem();  // the MMAs read dS^T through the async proxy
      tc_fence_before();
      mbar_arrive(B(bars->p_full[w]));
      // this half's dQ^T: read it, hand the columns back, add it into the accumulator
      ok = mbar_wait(B(bars->dq_full[w]), t & 1, wc);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      tc_fence_after();
      uint32_t dq[32];
      tmem_ld32(t_lane + 128 + c_s, dq);
      tmem_ld_wait<32>(dq);
      tc_fence_before();
      mbar_arrive(B(bars->dq_read[w]));
      if (dcol >= 0) {  // four rows of one element per reduction, 512 bytes per warp instruction
        const int rows = min(p.TPH, u.sq - tok0) * p.GS - 32 * sub;  // rows with a query
        float* acc = p.dqacc + (slot0 + i) * (kHalf * D) +
                     (static_cast<size_t>(8 * sub) * D + dcol) * 4;
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if (4 * e < rows)
            red_add_v4_f32(acc + static_cast<size_t>(e) * D * 4, dq[4 * e], dq[4 * e + 1],
                           dq[4 * e + 2], dq[4 * e + 3]);
      }
    }
    // epilogue of this thread's key: warpgroups 0, 1 write halves of dV, 2, 3 halves of dK
    if (ok) {
      ok = mbar_wait(B(bars->acc_full), 0, wc);
      ok = __all_sync(0xffffffffu, ok);
    }
    if (ok) {
      tc_fence_after();
      const bool is_k = grp >= 2;
      const float mul = is_k && p.HS == 1 ? p.scale : 1.f;
      const int64_t krow = u.k0 + row;
      const int c_lo = (grp % 2) * (D / 64);
#pragma unroll 1
      for (int c = c_lo; c < c_lo + D / 64; ++c) {
        uint32_t v[32];
        tmem_ld32(t_lane + 256 + (is_k ? D : 0) + c * 32, v);
        tmem_ld_wait<32>(v);
        if (u.n == 0) {  // no query sees these keys: zeros, not TMEM contents
#pragma unroll
          for (int e = 0; e < 32; ++e) v[e] = 0u;
        }
        if (row < u.nk) {
          if (p.HS > 1) {
            const size_t plane = static_cast<size_t>(p.total_k) * p.Hkv * D;
            uint4* dst = reinterpret_cast<uint4*>(
                p.part + (2 * static_cast<size_t>(hh - kvh * p.HS) + (is_k ? 0 : 1)) * plane +
                (static_cast<size_t>(krow) * p.Hkv + kvh) * D + c * 32);
#pragma unroll
            for (int e = 0; e < 8; ++e)
              dst[e] = make_uint4(v[4 * e], v[4 * e + 1], v[4 * e + 2], v[4 * e + 3]);
          } else {
            uint32_t pk[16];
#pragma unroll
            for (int e = 0; e < 16; ++e) {
              const float a = __uint_as_float(v[2 * e]) * mul, b = __uint_as_float(v[2 * e + 1]) * mul;
              pk[e] = BF16 ? cvt_pack_bf16(a, b) : cvt_pack_f16(a, b);
            }
            uint4* dst = reinterpret_cast<uint4*>(
                static_cast<uint16_t*>(is_k ? p.dk : p.dv) +
                krow * (is_k ? p.dk_token : p.dv_token) + kvh * D + c * 32);
#pragma unroll
            for (int e = 0; e < 4; ++e)
              dst[e] = make_uint4(pk[4 * e], pk[4 * e + 1], pk[4 * e + 2], pk[4 * e + 3]);
          }
        }
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 0) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

template <int D, bool BF16>
cudaError_t launch_t(const VarBwdLaunch& L, cudaStream_t stream) {
  const VarBwdParams& p = L.p;
  const int per = p.Hkv * p.HS;
  cudaError_t e;
  const dim3 slots(p.slots, per);
  const dim3 prep = p.total_q > 0 ? dim3(p.slots + 1, per) : dim3(1, 1);  // CTA (0, 0) plans
  bwd_prep_kernel<D, BF16><<<prep, kPrepThreads, 0, stream>>>(p);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  if (p.total_k > 0) {
    constexpr int smem = Cfg<D>::SMEM;
    auto* k = bwd_main_kernel<D, BF16>;
    e = prepare_kernel<bwd_main_kernel<D, BF16>>(smem);
    if (e != cudaSuccess) return e;
    k<<<static_cast<unsigned>(p.max_units) * per, kThreads, smem, stream>>>(L.tmQ, L.tmK, L.tmV,
                                                                            L.tmdO, p);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    if (p.HS > 1) {
      bwd_sum_kernel<D, BF16><<<dim3(4 * p.max_units, p.Hkv), 256, 0, stream>>>(p);
      if ((e = cudaGetLastError()) != cudaSuccess) return e;
    }
  }
  if (p.total_q > 0) {  // without keys the accumulator stays 0 and so does dq
    bwd_dq_kernel<D, BF16><<<slots, 256, 0, stream>>>(p);
    e = cudaGetLastError();
  }
  return e;
}

}  // namespace

cudaError_t launch_bwd_varlen(const VarBwdLaunch& L, int D, bool bf16, cudaStream_t stream) {
  if (D == 128) return bf16 ? launch_t<128, true>(L, stream) : launch_t<128, false>(L, stream);
  return bf16 ? launch_t<64, true>(L, stream) : launch_t<64, false>(L, stream);
}

}  // namespace fa
