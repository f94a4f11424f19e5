// Internal interface between the C-ABI layer (fa_api_varlen.cu) and the kernels over packed
// tokens: rotary positions, packed grouped-head attention, its gradient, and attention of new
// tokens over a paged cache.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <atomic>
#include <cstddef>
#include <cstdint>

#include "fa.h"
#include "fa_internal.h"

namespace fa {

// The dynamic shared memory of KERN, set once per device (a driver call otherwise paid per call).
template <auto KERN>
inline cudaError_t prepare_kernel(int smem) {
  static std::atomic<uint64_t> ready{0};  // this kernel: one bit per device index below 64
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = dev < 64 ? uint64_t{1} << dev : 0;
  if (bit && (ready.load(std::memory_order_acquire) & bit)) return cudaSuccess;
  e = cudaFuncSetAttribute(KERN, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e == cudaSuccess) ready.fetch_or(bit, std::memory_order_release);
  return e;
}

// Rotary positions (fa_rope.cu). Token and head steps are in elements. fa_rope: x -> y, H
// heads, pos[T]. fa_rope_append: x = q and y = q_out with heads d apart, k and v beside it,
// positions from ctx and cu, k and v into the pools.
struct RopeParams {
  const void* x;
  void* y;
  const double* freqs;  // [rot/2] radians per position
  const int32_t* pos;
  int64_t T, x_token, x_head, y_token, y_head;
  int H, d, rot;
  float amplitude;
  int inverse, copy_rest;  // copy_rest: elements rot .. d-1 are copied (not when y is x)
  const void* k;
  const void* v;
  void* k_pages;
  void* v_pages;
  int64_t k_token, v_token;
  const int32_t* cu;           // [B+1]
  const int32_t* ctx;          // [B] tokens cached before the chunk
  const int32_t* block_table;  // [B, max_pages]
  int B, Hkv, page_size, max_pages, num_pages;
  uint32_t* status;
};
cudaError_t launch_rope(const RopeParams& p, int dtype, bool half_style, bool vec, int sms,
                        cudaStream_t stream);
cudaError_t launch_rope_append(const RopeParams& p, int dtype, bool half_style, bool vec, int sms,
                               cudaStream_t stream);

// Norms of query and key heads with rotary positions (fa_norm_rope.cu). Token and head steps are
// in elements. Rows of a token: H of q, Hkv of k and, when appending, Hkv of v.
struct NormRopeParams {
  const void* q;
  const void* k;
  const void* v;  // appending
  void* q_out;    // the gradient writes dq and dk here
  void* k_out;
  int64_t q_token, q_head, k_token, k_head, v_token;
  int64_t q_out_token, q_out_head, k_out_token, k_out_head;
  const double* freqs;       // [rot/2] radians per position
  const int32_t* pos;        // [axes][T]; appending: nullptr for the tokens' places
  const int32_t* pair_axis;  // [rot/2], or nullptr: axis 0
  const void* q_weight;      // [d] of the dtype, or of FP32 where w_f32; nullptr: ones
  const void* k_weight;
  int64_t T;
  int H, Hkv, d, rot, axes, norm, inverse, w_f32;
  float amplitude, eps;
  // appending
  void* k_pages;
  void* v_pages;
  uint8_t* k_scales;  // exponent bytes [num_pages, Hkv, page_size]; nullptr: 16-bit pools
  uint8_t* v_scales;
  const int32_t* cu;           // [B+1]
  const int32_t* ctx;          // [B] tokens cached before the chunk
  const int32_t* block_table;  // [B, max_pages]
  int B, page_size, max_pages, num_pages;
  // gradient
  const void* dyq;
  const void* dyk;
  int64_t dyq_token, dyq_head, dyk_token, dyk_head;
  float* part;  // [CTAs][2][d] sums of the weights' gradients, or nullptr
  float* dq_weight;
  float* dk_weight;
  uint32_t* status;
};
constexpr int kNormCtas = 320;  // CTAs of the gradient at most, unless a token's heads need more
inline int norm_parts(int rows) { return rows / 8 > kNormCtas ? rows / 8 : kNormCtas; }
cudaError_t launch_norm_rope(const NormRopeParams& p, int dtype, bool half_style, bool vec,
                             int sms, cudaStream_t stream);
cudaError_t launch_norm_rope_bwd(const NormRopeParams& p, int dtype, bool half_style, bool vec,
                                 int sms, cudaStream_t stream);
cudaError_t launch_norm_rope_append(const NormRopeParams& p, int dtype, bool half_style, bool vec,
                                    int sms, cudaStream_t stream);

// Rows of an 8-bit cache back in 16 bits: tokens [cu[b], cu[b+1]) from position starts[b] on.
struct KvReadParams {
  const void* k_pages;  // [num_pages, Hkv, page_size, d]
  const void* v_pages;
  const uint8_t* k_scales;
  const uint8_t* v_scales;
  const int32_t* block_table;
  const int32_t* starts;
  const int32_t* cu;
  void* k;  // [T, Hkv, d]
  void* v;
  int64_t k_token, v_token, T;
  int B, Hkv, d, page_size, max_pages, num_pages;
  uint32_t* status;
};
cudaError_t launch_kv_read(const KvReadParams& p, bool bf16, int sms, cudaStream_t stream);

// ------------------------------------------------ packed grouped-head attention (fa_varlen.cu)
//
// Query heads come in groups of G = H / Hkv that read the same K/V head. A tensor-core tile of
// 128 rows holds TPT = 128 / G consecutive tokens with the G heads of one group (row r: token
// r / G, head r % G of the group); a work item is two such tiles, 2 TPT tokens, over a run of
// the key blocks that they see.

constexpr int kVarBN = 128;  // keys per block

// One work item of every K/V head, written by the plan kernel (48 bytes).
struct VarUnit {
  int32_t q0, nq;  // first row of q, tokens (<= 2 TPT)
  int32_t sk, k0;  // keys of the sequence; its first row of k and v
  int32_t qpos;    // key position of the first token (queries are the last of the keys)
  int32_t seq;
  int32_t j0, j1;  // which of the visited key blocks
  int32_t slot;    // -1: writes o and lse; else a partial result, slot * Hkv + kv head
  int32_t a_end, b_start;  // visited blocks: 0 .. a_end - 1, then b_start on
  int32_t start;   // key position of the sequence's first token
};
// A token block whose key blocks were split: its partial results, slot .. slot + n - 1.
struct VarGroup {
  int32_t q0, nq, slot, n;
};
struct VarHeader {
  int32_t units, groups, pad[14];
};

constexpr int kVarMaxSplit = 456;  // work items (all K/V heads) of a split plan: 3 per SM
constexpr int kVarSplitRows = 256;
inline size_t var_slot_floats(int d) { return static_cast<size_t>(kVarSplitRows) * (d + 2); }

struct VarParams {
  PrefillParams m;  // mask_mode, window, n_global, sl2, status, timeout_ns alone are read
  void* o;          // [total_q, H, D], o_token elements from one token to the next
  float* lse;       // [total_q, H] or nullptr
  int64_t o_token;
  int B, H, Hkv, G, TPT, total_q, total_k;
  const int32_t* cu_q;  // [B+1]
  const int32_t* cu_k;  // [B+1] (contiguous K/V)
  // paged K/V: lengths and table; a key block is loaded as boxes of `box` rows of one page
  const int32_t* ctx;
  const int32_t* block_table;
  int page_size, max_pages, num_pages, box;
  // an 8-bit cache: pools and exponent bytes; null otherwise
  const void* k_pages;
  const void* v_pages;
  const uint8_t* k_scales;
  const uint8_t* v_scales;
  const uint32_t* tree;  // FA_MASK_TREE: [total_q][tree_words]
  int tree_words;
  // workspace
  VarHeader* hdr;
  VarUnit* units;
  VarGroup* groups;
  float* part;    // slots, or nullptr: no splitting
  int max_units;  // entries of `units`
  int cost_shift; // key blocks >> cost_shift is a sort key below 1024
};

struct VarLaunch {
  CUtensorMap tmQ, tmK, tmV, tmO;
  VarParams p;
  int sms;
  bool runs;  // the plan may cut the items into equal runs (fa_varlen.cu)
};
cudaError_t launch_varlen(const VarLaunch& L, int D, bool bf16, cudaStream_t stream);

// ------------------------------------------------ gradient (fa_varlen_bwd.cu)
//
// The query side moves in halves of 64 rows: TPH = 64 / GS consecutive tokens of a sequence with
// GS heads of one group (row r: token r / GS, head r % GS). A group's G heads are dealt to HS
// subsets of GS = G / HS when few key blocks would keep few SMs busy for long; each subset then
// has its own partial dk and dv. A half's slot in the dq accumulator: sequence b's halves start at
// cu[b] / TPH + b, which leaves room for every sequence's rounding without a scan (where a start is
// bad, the plan deals slots out instead).
constexpr int kBwdHalf = 64;

struct VarBwdUnit {  // one block of 128 keys (48 bytes), written by the plan kernel
  int32_t k0, nk, j0;     // first row of k, keys in the block, first key's position
  int32_t q0, sq, delta;  // first row of q, queries, sk - sq
  int32_t h0, n;          // halves that see a key of the block: h0 .. h0 + n - 1
  int32_t slot0, pad[3];  // slot of the sequence's first half
};

struct VarBwdParams {
  PrefillParams m;  // mask_mode, window, n_global, sl2, status, timeout_ns alone are read
  const void* o;
  const void* dout;
  const float* lse;
  void* dq;
  void* dk;
  void* dv;
  int64_t o_token, dout_token, dq_token, dk_token, dv_token;
  const int32_t* cu_q;
  const int32_t* cu_k;
  float scale;
  int B, H, Hkv, G, GS, HS, TPH, total_q, total_k;
  int slots;      // half slots: total_q / TPH + B + 1
  int max_units;  // entries of `units`
  int cost_shift;
  // workspace
  int32_t* n_units;   // [16]: units; whether the slots were dealt out
  VarBwdUnit* units;
  int32_t* seq_slot;  // [B]: first slot of the sequence or -1, where slots were dealt out
  float* stats;       // [2][Hkv HS][total_q][GS]: -lse log2(e), -D; a half behind them is read
  float* dqacc;       // [Hkv HS][slots][16 groups of 4 rows][D][4]
  float* part;        // HS > 1: [HS][2 (dk, dv)][total_k][Hkv][D]
};

struct VarBwdLaunch {
  CUtensorMap tmQ, tmK, tmV, tmdO;
  VarBwdParams p;
};
cudaError_t launch_bwd_varlen(const VarBwdLaunch& L, int D, bool bf16, cudaStream_t stream);

// ------------------------------------------------ few rows over a paged cache (fa_few.cu)
//
// Chunks whose rows (tokens x heads of a group) are at most 16, a decode step above all: bound
// by reading the cache, so the key tiles of all sequences and K/V heads are laid end to end and
// dealt to the CTAs in equal runs, whatever the lengths.
constexpr int kFewRows = 16;
constexpr int kFewMaxCtas = 320;
// A pair (sequence, K/V head) whose first piece CTA x holds: its first row of q, rows, K/V head,
// and the CTA of its last piece; rows = 0: none.
struct FewHead {
  int32_t q0, rows, kvh, last;
};
constexpr size_t kFewHeadBytes = kFewMaxCtas * sizeof(FewHead);
inline size_t few_part_floats(int d) {  // a CTA leaves at most two partial results
  return static_cast<size_t>(2) * kFewMaxCtas * kFewRows * (d + 2);
}

struct FewParams {
  PrefillParams m;  // mask_mode, window, n_global, sl2, status, timeout_ns alone are read
  const void* q;
  void* o;
  float* lse;
  int64_t q_token, o_token;
  const int32_t* cu_q;
  const int32_t* ctx;
  const int32_t* block_table;
  int B, H, Hkv, G, total_q, max_q;
  int page_size, max_pages, num_pages, box;  // box: rows of one TMA box (<= 64, 8 bits 128)
  const uint8_t* k_scales;  // exponent bytes of an 8-bit cache [num_pages, Hkv, page_size], or null
  const uint8_t* v_scales;
  const uint32_t* tree;  // FA_MASK_TREE: [total_q][tree_words]
  int tree_words;
  FewHead* heads;  // [CTAs]
  float* part;  // [2 CTAs][16 rows][D], then m [2 CTAs][16], l [2 CTAs][16] (or 8 rows: fa_few8.cu)
};

struct FewLaunch {
  CUtensorMap tmK, tmV;
  FewParams p;
  int sms;
};
cudaError_t launch_few(const FewLaunch& L, int D, bool bf16, cudaStream_t stream);
// The same over an 8-bit cache (fa_few8.cu). With at most 8 rows it has more CTAs, whose pieces have 8
// rows each and fit in the same workspace.
constexpr int kFew8MaxCtas = 480;
constexpr int kFew8Blocks = 2;                // blocks of 16 keys of a warp
constexpr int kFew8Tile = 64 * kFew8Blocks;   // keys of a tile
constexpr size_t kFew8HeadBytes = kFew8MaxCtas * sizeof(FewHead);
static_assert(kFew8HeadBytes + 2 * kFew8MaxCtas * 8 * (64 + 2) * 4 <=
                  kFewHeadBytes + 2 * kFewMaxCtas * kFewRows * (64 + 2) * 4 &&
              kFew8HeadBytes + 2 * kFew8MaxCtas * 8 * (128 + 2) * 4 <=
                  kFewHeadBytes + 2 * kFewMaxCtas * kFewRows * (128 + 2) * 4,
              "over the workspace");
cudaError_t launch_few8(const FewLaunch& L, int D, bool bf16, cudaStream_t stream);

}  // namespace fa
