// What the plan kernels of the packed calls share: one CTA reads the sequences' lengths on the
// device, visits every part (a block of queries or keys) of every sequence, and sorts the parts
// by cost with a counting sort, most expensive first.
#pragma once

#include <cstdint>

#include "fa_varlen.h"

namespace fa {
namespace {

constexpr int kPlanThreads = 1024;  // of the forward's plan; NT below: threads of the CTA
constexpr int kBins = 1024;

// One sequence: first rows and lengths of its queries and keys, and its number of parts.
struct Seq {
  int q0, sq, k0, sk, parts;
};

template <int NT>
struct SeqScan {
  static_assert(NT % 32 == 0 && NT <= 1024 && kBins % NT == 0, "whole warps, a share of the bins");
  int off[NT + 1];  // parts before each sequence of the batch
  Seq seq[NT];
  int warp_sum[NT / 32];
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

// Inclusive scan over the CTA's threads (every thread takes part; `sums` is scratch of one word
// per warp, which holds the inclusive scan of the warps' sums afterwards).
template <int NT>
__device__ __forceinline__ int scan_cta(int x, int* sums) {
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  for (int o = 1; o < 32; o *= 2) {
    const int y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) sums[warp] = x;
  __syncthreads();
  if (warp == 0) {
    int w = lane < NT / 32 ? sums[lane] : 0;
    for (int o = 1; o < 32; o *= 2) {
      const int y = __shfl_up_sync(0xffffffffu, w, o);
      if (lane >= o) w += y;
    }
    if (lane < NT / 32) sums[lane] = w;
  }
  __syncthreads();
  return x + (warp ? sums[warp - 1] : 0);
}

// load(b) -> Seq for every sequence, f(b, seq, part) for every part of every sequence;
// sequences go in batches of one per thread. Every thread of the CTA takes part.
template <int NT, typename Load, typename F>
__device__ __forceinline__ void for_each_part(SeqScan<NT>& s, int B, Load load, F f) {
  const int tid = threadIdx.x;
  for (int base = 0; base < B; base += NT) {
    Seq q{0, 0, 0, 0, 0};
    if (base + tid < B) {
      q = load(base + tid);
      s.seq[tid] = q;
    }
    const int upto = scan_cta<NT>(q.parts, s.warp_sum);
    s.off[tid + 1] = upto;
    if (tid == 0) s.off[0] = 0;
    __syncthreads();
    const int n = min(NT, B - base), total = s.off[n];
    for (int i = tid; i < total; i += NT) {
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
template <int NT>
__device__ __forceinline__ int scan_bins(SeqScan<NT>& s, int* bins) {
  constexpr int PER = kBins / NT;  // bins of a thread
  int v[PER], sum = 0;
#pragma unroll
  for (int i = 0; i < PER; ++i) sum += v[i] = bins[threadIdx.x * PER + i + 1];
  int at = scan_cta<NT>(sum, s.warp_sum) - sum;  // (its barriers part the reads from the writes)
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    bins[threadIdx.x * PER + i] = at;
    at += v[i];
  }
  __syncthreads();
  const int all = s.warp_sum[NT / 32 - 1];
  __syncthreads();
  return all;
}

}  // namespace
}  // namespace fa
