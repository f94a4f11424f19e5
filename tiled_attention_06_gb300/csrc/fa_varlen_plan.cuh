// What the plan kernels of the packed calls share: one CTA reads the sequences' lengths on the
// device, visits every part (a block of queries or keys) of every sequence, and sorts the parts
// by cost with a counting sort, most expensive first.
#pragma once

#include <cstdint>

#include "fa_varlen.h"

namespace fa {
namespace {

constexpr int kPlanThreads = 1024;
constexpr int kBins = 1024;
static_assert(kBins == kPlanThreads, "the scan takes one bin per thread");
static_assert(kPlanThreads == 32 * 32, "the scan reads a sum of every one of 32 warps");

// One sequence: first rows and lengths of its queries and keys, and its number of parts.
struct Seq {
  int q0, sq, k0, sk, parts;
};

struct SeqScan {
  int off[kPlanThreads + 1];  // parts before each sequence of the batch
  Seq seq[kPlanThreads];
  int warp_sum[32];
};

// Rows [first, first + n) of sequence b, empty when its starts make no sense.
struct SeqRows {
  int first, n;
  bool bad;
};
__device__ __forceinline__ SeqRows rows_of(const int32_t* cu, int b, int total) {
  const int a = cu[b], e = cu[b + 1];
  const bool bad = a < 0 || e < a || e > total;
  return SeqRows{bad ? 0 : a, bad ? 0 : e - a, bad};
}

// Inclusive scan over the CTA's threads (every thread takes part; `sums` is scratch).
__device__ __forceinline__ int scan_cta(int x, int* sums) {
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  for (int o = 1; o < 32; o *= 2) {
    const int y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) sums[warp] = x;
  __syncthreads();
  if (warp == 0) {
    int w = sums[lane];
    for (int o = 1; o < 32; o *= 2) {
      const int y = __shfl_up_sync(0xffffffffu, w, o);
      if (lane >= o) w += y;
    }
    sums[lane] = w;
  }
  __syncthreads();
  return x + (warp ? sums[warp - 1] : 0);
}

// load(b) -> Seq for every sequence, f(b, seq, part) for every part of every sequence;
// sequences go in batches of one per thread. Every thread of the CTA takes part.
template <typename Load, typename F>
__device__ __forceinline__ void for_each_part(SeqScan& s, int B, Load load, F f) {
  const int tid = threadIdx.x;
  for (int base = 0; base < B; base += kPlanThreads) {
    Seq q{0, 0, 0, 0, 0};
    if (base + tid < B) {
      q = load(base + tid);
      s.seq[tid] = q;
    }
    const int upto = scan_cta(q.parts, s.warp_sum);
    s.off[tid + 1] = upto;
    if (tid == 0) s.off[0] = 0;
    __syncthreads();
    const int n = min(kPlanThreads, B - base), total = s.off[n];
    for (int i = tid; i < total; i += kPlanThreads) {
      int lo = 0, hi = n;  // the last sequence that starts at or before part i
      while (hi - lo > 1) {
        const int mid = (lo + hi) / 2;
        if (s.off[mid] <= i)
          lo = mid;
        else
          hi = mid;
      }
      f(base + lo, s.seq[lo], i - s.off[lo]);
    }
    __syncthreads();
  }
}

__device__ __forceinline__ int cost_bin(int n, int shift) {
  return kBins - 1 - min(kBins - 1, n >> shift);  // the most expensive first
}

// bins[i + 1] holds the number of parts of bin i; afterwards bins[i] is the place of the first
// of them. Returns the number of all.
__device__ __forceinline__ int scan_bins(SeqScan& s, int* bins) {
  const int v = bins[threadIdx.x + 1];
  const int upto = scan_cta(v, s.warp_sum);
  __syncthreads();
  bins[threadIdx.x] = upto - v;
  __syncthreads();
  const int all = s.warp_sum[31];
  __syncthreads();
  return all;
}

}  // namespace
}  // namespace fa
