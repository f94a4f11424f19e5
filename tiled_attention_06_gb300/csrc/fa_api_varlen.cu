// The C ABI of the calls over packed tokens (include/fa.h): rotary positions, packed
// grouped-head attention and its gradient, attention of new tokens over a paged cache.
// Every check runs on the host before anything is launched.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstring>

#include "fa.h"
#include "fa_host.h"
#include "fa_varlen.h"

namespace {

using fa::host::aligned16;
using fa::host::aligned4;
using fa::host::check_packed;
using fa::host::cuda_fail;
using fa::host::device_info;
using fa::host::DeviceInfo;
using fa::host::encode_fn;
using fa::host::fail;

constexpr double kTwoPi = 6.283185307179586476925286766559;

bool aligned8(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 7u) == 0; }
size_t round16(size_t n) { return (n + 15) / 16 * 16; }
size_t round256(size_t n) { return (n + 255) / 256 * 256; }
int ceil_div(long long a, long long b) { return static_cast<int>((a + b - 1) / b); }

// A 16-bit tensor of three dimensions (the first of `d` contiguous elements) as a TMA map with
// 128-byte swizzle; strides in elements, one box is 64 x box1 x box2.
fa_status make_map3(CUtensorMap* m, const void* ptr, bool bf16, int d, long long n1, long long s1,
                    long long n2, long long s2, int box1, int box2) {
  auto enc = encode_fn();
  if (!enc) return fail(FA_ERR_CUDA, "cuTensorMapEncodeTiled is not available from the driver");
  const cuuint64_t dims[3] = {static_cast<cuuint64_t>(d), static_cast<cuuint64_t>(n1),
                              static_cast<cuuint64_t>(n2)};
  const cuuint64_t strides[2] = {static_cast<cuuint64_t>(s1) * 2, static_cast<cuuint64_t>(s2) * 2};
  const cuuint32_t box[3] = {64, static_cast<cuuint32_t>(box1), static_cast<cuuint32_t>(box2)};
  const cuuint32_t estr[3] = {1, 1, 1};
  const CUresult r = enc(
      m, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3,
      const_cast<void*>(ptr), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
      CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
      CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) return fail(FA_ERR_CUDA, "cuTensorMapEncodeTiled failed (%d)", (int)r);
  return FA_OK;
}

// Rows of d bytes of an 8-bit cache, (d, page_size, planes): boxes of whole rows, swizzled over
// them.
fa_status make_map8(CUtensorMap* m, const void* ptr, int d, int page_size, long long planes,
                    int box) {
  auto enc = encode_fn();
  if (!enc) return fail(FA_ERR_CUDA, "cuTensorMapEncodeTiled is not available from the driver");
  const cuuint64_t dims[3] = {static_cast<cuuint64_t>(d), static_cast<cuuint64_t>(page_size),
                              static_cast<cuuint64_t>(planes)};
  const cuuint64_t strides[2] = {static_cast<cuuint64_t>(d),
                                 static_cast<cuuint64_t>(d) * page_size};
  const cuuint32_t boxes[3] = {static_cast<cuuint32_t>(d), static_cast<cuuint32_t>(box), 1};
  const cuuint32_t estr[3] = {1, 1, 1};
  const CUresult r =
      enc(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<void*>(ptr), dims, strides, boxes, estr,
          CU_TENSOR_MAP_INTERLEAVE_NONE,
          d == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
          CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) return fail(FA_ERR_CUDA, "cuTensorMapEncodeTiled failed (%d)", (int)r);
  return FA_OK;
}

// What every attention call here has in common.
struct Common {
  int B, H, Hkv, d, total_q;
  float scale;
  int mask_mode, window, n_global, dtype;
};

fa_status check_common(const Common& c) {
  if (c.B < 1 || c.H < 1 || c.Hkv < 1 || c.total_q < 0)
    return fail(FA_ERR_INVALID_ARG, "need B, H, Hkv >= 1 and total_q >= 0");
  if (c.H % c.Hkv != 0)
    return fail(FA_ERR_INVALID_ARG, "H = %d is not a multiple of Hkv = %d", c.H, c.Hkv);
  if (c.H / c.Hkv > 128)
    return fail(FA_ERR_UNSUPPORTED, "%d query heads per K/V head (at most 128)", c.H / c.Hkv);
  if (c.d != 64 && c.d != 128)
    return fail(FA_ERR_UNSUPPORTED, "head dim %d (supported: 64, 128)", c.d);
  if (c.dtype != FA_F16 && c.dtype != FA_BF16) return fail(FA_ERR_UNSUPPORTED, "dtype %d", c.dtype);
  // hidden scores are -inf before the scale is applied, and the maximum is taken unscaled
  if (!(c.scale > 0) || !std::isfinite(c.scale))
    return fail(FA_ERR_INVALID_ARG, "scale must be positive and finite");
  if (c.mask_mode < FA_MASK_NONE || c.mask_mode > FA_MASK_BLOCK_SPARSE)
    return fail(FA_ERR_INVALID_ARG, "mask_mode %d", c.mask_mode);
  if (c.mask_mode == FA_MASK_BLOCK_SPARSE)
    return fail(FA_ERR_UNSUPPORTED, "packed sequences take no block layout");
  if (c.mask_mode == FA_MASK_CAUSAL_WINDOW && (c.window < 1 || c.n_global < 0))
    return fail(FA_ERR_INVALID_ARG, "CAUSAL_WINDOW needs window >= 1 and n_global >= 0");
  if (c.mask_mode == FA_MASK_BAND && c.window < 0)
    return fail(FA_ERR_INVALID_ARG, "BAND needs window >= 0");
  if (c.mask_mode == FA_MASK_PREFIX_LM && c.n_global < 0)
    return fail(FA_ERR_INVALID_ARG, "PREFIX_LM needs n_global >= 0");
  if (c.B > (1 << 24) || c.H > (1 << 16) || c.total_q > (1 << 30) ||
      static_cast<long long>(c.total_q) * c.H > (1LL << 31) - 1)
    return fail(FA_ERR_INVALID_ARG, "problem too large");
  return FA_OK;
}

// Work items (per K/V head) that the plan of these sizes may hold without splitting, and
// whether there can be so few that it splits them.
int var_pairs(int B, int G, int total_q) {
  const int tpi = 2 * (128 / G);
  const long long n = static_cast<long long>(total_q) / tpi + B;
  return static_cast<int>(std::min<long long>(n, std::max(total_q, 1)));
}
bool var_may_split(int G, int Hkv, int total_q) {
  return static_cast<long long>(ceil_div(std::max(total_q, 1), 2 * (128 / G))) * Hkv <
         fa::kVarMaxSplit;
}

struct VarLayout {
  size_t hdr, units, groups, part, total;
  int max_units;
  bool split;
};
VarLayout var_layout(int B, int H, int Hkv, int total_q, int d) {
  VarLayout L;
  const int G = H / Hkv;
  L.split = var_may_split(G, Hkv, total_q);
  L.max_units = var_pairs(B, G, total_q);
  if (L.split) L.max_units = std::max(L.max_units, fa::kVarMaxSplit / Hkv);
  L.hdr = 0;
  L.units = round16(sizeof(fa::VarHeader));
  L.groups = L.units + round16(sizeof(fa::VarUnit) * static_cast<size_t>(L.max_units));
  L.part = L.groups + round16(L.split ? sizeof(fa::VarGroup) * fa::kVarMaxSplit : 0);
  L.total = L.part + (L.split ? fa::kVarMaxSplit * fa::var_slot_floats(d) * sizeof(float) : 0);
  return L;
}

// How the backward deals a group's heads and lays its workspace out (fa_varlen.h).
struct BwdLayout {
  int HS, GS, TPH, slots, max_units;
  size_t units, seq_slot, stats, dqacc, part, total;
};
BwdLayout bwd_layout(int B, int H, int Hkv, int total_q, int total_k, int d) {
  BwdLayout L;
  const int G = H / Hkv;
  // The divisor of G with the least time to expect. Key blocks: every sequence leaves half a
  // block on average. A CTA takes about 9 us around its halves of 64 rows and 1.1 us (0.6 at
  // d = 64) for each; under a causal mask a block sees half the queries on average and the first
  // block all of them. Subsets cost a summing pass (5 us, and their partials at 4 TB/s).
  // One sequence of 4096, 8 heads on one: HS = 8 took 137 us, 4 took 210; 24 short ones of
  // d = 64, 12 heads on 4: HS = 1 took 44 us, 3 took 61 (measured when the plan was a launch of
  // 5 us before all four). 152 is the number of SMs of a GB300, a constant so that the workspace
  // has one size wherever it is asked for; another count would change the time alone.
  const double units = (total_k / 128 + (B + 1) / 2) * static_cast<double>(Hkv);
  const double all = static_cast<double>(total_q) / B * G / fa::kBwdHalf;
  const double each = d == 128 ? 1.1 : 0.6;
  double best = 0;
  L.HS = 0;
  for (int hs = 1; hs <= G; ++hs) {
    if (G % hs || G / hs > fa::kBwdHalf) continue;
    const double t =
        std::max(9.0 + all / hs * each, units * hs / 152 * (9.0 + 0.5 * all / hs * each)) +
        (hs > 1 ? 5.0 + static_cast<double>(hs) * total_k * Hkv * d * 8 / 4e6 : 0.0);
    if (!L.HS || t < best) {
      best = t;
      L.HS = hs;
    }
  }
  L.GS = G / L.HS;
  L.TPH = fa::kBwdHalf / L.GS;
  L.slots = total_q / L.TPH + B + 1;
  L.max_units = static_cast<int>(
      std::min<long long>(static_cast<long long>(total_k) / 128 + B, std::max(total_k, 1)));
  const size_t planes = static_cast<size_t>(Hkv) * L.HS * L.slots;
  L.units = 64;
  L.seq_slot = L.units + round16(sizeof(fa::VarBwdUnit) * static_cast<size_t>(L.max_units));
  // from here on whole cache lines: with the accumulator 16 bytes off one, 11343 tokens in 4
  // sequences took 806 us instead of 784
  L.stats = round256(L.seq_slot + sizeof(int32_t) * static_cast<size_t>(B));
  L.dqacc = round256(L.stats +
                     (2 * static_cast<size_t>(total_q) * H + fa::kBwdHalf) * sizeof(float));
  L.part = L.dqacc + planes * fa::kBwdHalf * d * sizeof(float);
  L.total = L.part + (L.HS > 1 ? static_cast<size_t>(L.HS) * 2 * total_k * Hkv * d * sizeof(float)
                               : 0);
  return L;
}

// Chunks of up to max_q tokens are few rows (fa_few.cu).
bool few_rows(int max_q, int G) {
  return static_cast<long long>(std::max(max_q, 1)) * G <= fa::kFewRows;
}

fa_status check_workspace(const void* ws, size_t bytes, size_t need) {
  if (!ws || !aligned16(ws))
    return fail(FA_ERR_INVALID_ARG, "a 16-byte aligned workspace is needed");
  if (bytes < need)
    return fail(FA_ERR_INVALID_ARG, "workspace has %zu bytes, needs %zu", bytes, need);
  return FA_OK;
}

void fill_mask(fa::PrefillParams* m, const Common& c, uint32_t timeout_us, uint32_t* status) {
  const bool w = c.mask_mode == FA_MASK_CAUSAL_WINDOW || c.mask_mode == FA_MASK_BAND;
  const bool g = c.mask_mode == FA_MASK_CAUSAL_WINDOW || c.mask_mode == FA_MASK_PREFIX_LM;
  m->mask_mode = c.mask_mode;
  m->window = w ? std::min(c.window, fa::kMaxWindow) : 0;
  m->n_global = g ? std::min(c.n_global, 1 << 30) : 0;  // no sequence has more keys
  m->sl2 = c.scale * 1.4426950408889634f;
  m->status = status;
  m->timeout_ns = static_cast<uint64_t>(timeout_us ? timeout_us : 1000000u) * 1000u;
}

// Fields shared by the packed and the paged call.
void fill_var(fa::VarParams* p, const Common& c, void* o, float* lse, int64_t o_token,
              const int32_t* cu_q, void* workspace, long long max_keys, uint32_t timeout_us,
              uint32_t* status) {
  fill_mask(&p->m, c, timeout_us, status);
  p->o = o;
  p->lse = lse;
  p->o_token = o_token;
  p->B = c.B;
  p->H = c.H;
  p->Hkv = c.Hkv;
  p->G = c.H / c.Hkv;
  p->TPT = 128 / p->G;
  p->total_q = c.total_q;
  p->cu_q = cu_q;
  const VarLayout L = var_layout(c.B, c.H, c.Hkv, c.total_q, c.d);
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  p->hdr = reinterpret_cast<fa::VarHeader*>(ws + L.hdr);
  p->units = reinterpret_cast<fa::VarUnit*>(ws + L.units);
  p->groups = reinterpret_cast<fa::VarGroup*>(ws + L.groups);
  p->part = L.split ? reinterpret_cast<float*>(ws + L.part) : nullptr;
  p->max_units = L.max_units;
  p->cost_shift = 0;
  while (((max_keys / fa::kVarBN + 1) >> p->cost_shift) >= 1024) ++p->cost_shift;
}

}  // namespace

extern "C" {

fa_status fa_rope_freqs(double* freqs, float* amplitude, int rot_dim, double base, int scaling,
                        double factor, int trained_len, double fast, double slow) {
  if (!freqs || !amplitude)
    return fail(FA_ERR_INVALID_ARG, "freqs and amplitude must be non-null");
  if (rot_dim < 2 || rot_dim > 512 || rot_dim % 2)
    return fail(FA_ERR_INVALID_ARG, "rot_dim %d (even, in [2, 512])", rot_dim);
  if (scaling < FA_ROPE_PLAIN || scaling > FA_ROPE_BY_PARTS)
    return fail(FA_ERR_INVALID_ARG, "scaling %d", scaling);
  if (!(base > 0) || !std::isfinite(base)) return fail(FA_ERR_INVALID_ARG, "base must be positive");
  if (scaling != FA_ROPE_PLAIN && !(factor >= 1 && std::isfinite(factor)))
    return fail(FA_ERR_INVALID_ARG, "factor must be at least 1");
  if (scaling == FA_ROPE_BASE && rot_dim < 4)
    return fail(FA_ERR_INVALID_ARG, "FA_ROPE_BASE needs rot_dim >= 4");
  if (scaling == FA_ROPE_BY_PARTS && (trained_len < 1 || !(fast > slow) || !std::isfinite(fast) ||
                                      !std::isfinite(slow)))
    return fail(FA_ERR_INVALID_ARG, "FA_ROPE_BY_PARTS needs trained_len >= 1 and fast > slow");
  if (scaling == FA_ROPE_BASE)
    base *= std::pow(factor, static_cast<double>(rot_dim) / (rot_dim - 2));
  for (int i = 0; i < rot_dim / 2; ++i) {
    const double w = std::pow(base, -2.0 * i / rot_dim);
    if (scaling == FA_ROPE_LINEAR) {
      freqs[i] = w / factor;
    } else if (scaling == FA_ROPE_BY_PARTS) {
      const double r = trained_len * w / kTwoPi;
      const double g = std::min(1.0, std::max(0.0, (r - slow) / (fast - slow)));
      freqs[i] = g * w + (1.0 - g) * (w / factor);
    } else {
      freqs[i] = w;
    }
  }
  *amplitude =
      scaling == FA_ROPE_BY_PARTS ? static_cast<float>(0.1 * std::log(factor) + 1.0) : 1.f;
  return FA_OK;
}

fa_status fa_rope(const void* x, void* y, const int32_t* positions, const double* freqs, int64_t T,
                  int H, int d, int rot_dim, int64_t x_token, int64_t x_head, int64_t y_token,
                  int64_t y_head, int style, float amplitude, int inverse, int dtype,
                  fa_stream_t stream) {
  if (dtype != FA_F16 && dtype != FA_BF16 && dtype != FA_F32)
    return fail(FA_ERR_UNSUPPORTED, "dtype %d", dtype);
  if (T < 0 || H < 1 || d < 2 || d > 512)
    return fail(FA_ERR_INVALID_ARG, "need T >= 0, H >= 1 and d in [2, 512]");
  if (rot_dim < 2 || rot_dim > d || rot_dim % 2)
    return fail(FA_ERR_INVALID_ARG, "rot_dim %d (even, in [2, d])", rot_dim);
  if (d % 2) return fail(FA_ERR_UNSUPPORTED, "head dim %d (even)", d);
  if (style != FA_ROPE_HALF && style != FA_ROPE_PAIRS)
    return fail(FA_ERR_INVALID_ARG, "style %d", style);
  if (!std::isfinite(amplitude)) return fail(FA_ERR_INVALID_ARG, "amplitude must be finite");
  if (T == 0) return FA_OK;
  if (!x || !y || !positions || !freqs)
    return fail(FA_ERR_INVALID_ARG, "x, y, positions and freqs must be non-null");
  const size_t es = dtype == FA_F32 ? 4 : 2;
  const uintptr_t both = reinterpret_cast<uintptr_t>(x) | reinterpret_cast<uintptr_t>(y);
  if (both % es || !aligned4(positions) || !aligned8(freqs))
    return fail(FA_ERR_INVALID_ARG, "x, y, positions and freqs must be aligned to their elements");
  if (x_head < d || y_head < d || x_token < 0 || y_token < 0)
    return fail(FA_ERR_INVALID_ARG, "heads must be at least d elements apart, tokens not negative");
  const int64_t y_row = static_cast<int64_t>(H - 1) * y_head + d;
  if (T > 1 && y_token < y_row && !(y_head >= (T - 1) * y_token + d && y_token >= d))
    return fail(FA_ERR_INVALID_ARG, "the rows of y overlap");
  if (x == y && (x_token != y_token || x_head != y_head))
    return fail(FA_ERR_INVALID_ARG, "in place, x and y have the same steps");
  if (T > (1LL << 33) || static_cast<int64_t>(H) * d > (1LL << 28))
    return fail(FA_ERR_INVALID_ARG, "problem too large");
  DeviceInfo dev;
  const fa_status st = device_info(&dev);
  if (st != FA_OK) return st;
  fa::RopeParams p;
  std::memset(&p, 0, sizeof p);
  p.x = x;
  p.y = y;
  p.freqs = freqs;
  p.pos = positions;
  p.T = T;
  p.x_token = x_token;
  p.x_head = x_head;
  p.y_token = y_token;
  p.y_head = y_head;
  p.H = H;
  p.d = d;
  p.rot = rot_dim;
  p.amplitude = amplitude;
  p.inverse = inverse != 0;
  p.copy_rest = x != y;
  p.status = dev.status;
  const int v = static_cast<int>(16 / es);
  const bool vec = both % 16 == 0 && (x_token | x_head | y_token | y_head) % v == 0 &&
                   d % (2 * v) == 0 && rot_dim % (2 * v) == 0;
  const cudaError_t e = fa::launch_rope(p, dtype, style == FA_ROPE_HALF, vec, dev.sms,
                                        reinterpret_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "rope launch");
  return FA_OK;
}

fa_status fa_rope_append(const fa_rope_append_params* params, fa_stream_t stream) {
  if (!params) return fail(FA_ERR_INVALID_ARG, "params is null");
  const fa_rope_append_params& a = *params;
  if (a.dtype != FA_F16 && a.dtype != FA_BF16) return fail(FA_ERR_UNSUPPORTED, "dtype %d", a.dtype);
  if (a.T < 0 || a.B < 1 || a.H < 1 || a.Hkv < 1 || a.max_pages_per_seq < 1 || a.num_pages < 1)
    return fail(FA_ERR_INVALID_ARG,
                "need B, H, Hkv, max_pages_per_seq, num_pages >= 1 and T >= 0");
  if (a.d != 64 && a.d != 128)
    return fail(FA_ERR_UNSUPPORTED, "head dim %d (supported: 64, 128)", a.d);
  if (a.rot_dim < 2 || a.rot_dim > a.d || a.rot_dim % 2)
    return fail(FA_ERR_INVALID_ARG, "rot_dim %d (even, in [2, d])", a.rot_dim);
  if (a.page_size < 16 || a.page_size > 4096 || a.page_size % 16 != 0)
    return fail(FA_ERR_UNSUPPORTED, "page_size %d (a multiple of 16 in [16, 4096])", a.page_size);
  if (a.style != FA_ROPE_HALF && a.style != FA_ROPE_PAIRS)
    return fail(FA_ERR_INVALID_ARG, "style %d", a.style);
  if (!std::isfinite(a.amplitude)) return fail(FA_ERR_INVALID_ARG, "amplitude must be finite");
  if (a.H > (1 << 16) || a.Hkv > (1 << 16) ||
      static_cast<long long>(a.page_size) * a.max_pages_per_seq > (1LL << 30))
    return fail(FA_ERR_INVALID_ARG, "problem too large");
  if (a.T == 0) return FA_OK;
  fa_status st;
  if ((st = check_packed("q", a.q, a.q_token, a.H, a.d)) != FA_OK) return st;
  if ((st = check_packed("q_out", a.q_out, a.q_out_token, a.H, a.d)) != FA_OK) return st;
  if ((st = check_packed("k", a.k, a.k_token, a.Hkv, a.d)) != FA_OK) return st;
  if ((st = check_packed("v", a.v, a.v_token, a.Hkv, a.d)) != FA_OK) return st;
  if (a.q == a.q_out && a.q_token != a.q_out_token)
    return fail(FA_ERR_INVALID_ARG, "in place, q and q_out have the same step");
  if (!a.k_pages || !a.v_pages || !a.block_table || !a.ctx_lens || !a.cu_seqlens || !a.freqs)
    return fail(FA_ERR_INVALID_ARG,
                "pools, block_table, ctx_lens, cu_seqlens and freqs must be non-null");
  if (!aligned16(a.k_pages) || !aligned16(a.v_pages))
    return fail(FA_ERR_INVALID_ARG, "pools must be 16-byte aligned");
  if (!aligned4(a.block_table) || !aligned4(a.ctx_lens) || !aligned4(a.cu_seqlens) ||
      !aligned8(a.freqs))
    return fail(FA_ERR_INVALID_ARG, "integer arrays must be 4-byte aligned, freqs 8-byte");
  DeviceInfo dev;
  if ((st = device_info(&dev)) != FA_OK) return st;
  fa::RopeParams p;
  std::memset(&p, 0, sizeof p);
  p.x = a.q;
  p.y = a.q_out;
  p.freqs = a.freqs;
  p.T = a.T;
  p.x_token = a.q_token;
  p.y_token = a.q_out_token;
  p.x_head = p.y_head = a.d;
  p.H = a.H;
  p.d = a.d;
  p.rot = a.rot_dim;
  p.amplitude = a.amplitude;
  p.copy_rest = 1;
  p.k = a.k;
  p.v = a.v;
  p.k_pages = a.k_pages;
  p.v_pages = a.v_pages;
  p.k_token = a.k_token;
  p.v_token = a.v_token;
  p.cu = a.cu_seqlens;
  p.ctx = a.ctx_lens;
  p.block_table = a.block_table;
  p.B = a.B;
  p.Hkv = a.Hkv;
  p.page_size = a.page_size;
  p.max_pages = a.max_pages_per_seq;
  p.num_pages = a.num_pages;
  p.status = dev.status;
  const bool vec = a.rot_dim % 16 == 0;
  const cudaError_t e = fa::launch_rope_append(p, a.dtype, a.style == FA_ROPE_HALF, vec, dev.sms,
                                               reinterpret_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "rope append launch");
  return FA_OK;
}

size_t fa_varlen_workspace_size(int B, int H, int Hkv, int total_q, int total_k, int d) {
  (void)total_k;
  if (B < 1 || Hkv < 1 || H < Hkv || H % Hkv || H / Hkv > 128 || total_q < 0 || d < 1) return 0;
  return var_layout(B, H, Hkv, total_q, d).total;
}

static Common common_of(const fa_varlen_params& a) {
  return Common{a.B,         a.H,      a.Hkv,      a.d,    a.total_q, a.scale,
                a.mask_mode, a.window, a.n_global, a.dtype};
}

// Checks of the packed calls' inputs.
static fa_status check_varlen(const fa_varlen_params& a) {
  fa_status st = check_common(common_of(a));
  if (st != FA_OK) return st;
  if (a.total_k < 0 || a.total_k > (1 << 30) ||
      static_cast<long long>(a.total_k) * a.Hkv > (1LL << 31) - 1)
    return fail(FA_ERR_INVALID_ARG, "total_k %d", a.total_k);
  if (!a.cu_seqlens_q || !a.cu_seqlens_k || !aligned4(a.cu_seqlens_q) || !aligned4(a.cu_seqlens_k))
    return fail(FA_ERR_INVALID_ARG, "cu_seqlens_q and cu_seqlens_k: non-null, 4-byte aligned");
  if (a.total_q > 0) {
    if ((st = check_packed("q", a.q, a.q_token, a.H, a.d)) != FA_OK) return st;
    if ((st = check_packed("o", a.o, a.o_token, a.H, a.d)) != FA_OK) return st;
  }
  if (a.total_k > 0) {
    if ((st = check_packed("k", a.k, a.k_token, a.Hkv, a.d)) != FA_OK) return st;
    if ((st = check_packed("v", a.v, a.v_token, a.Hkv, a.d)) != FA_OK) return st;
  }
  if (!aligned4(a.lse)) return fail(FA_ERR_INVALID_ARG, "lse must be 4-byte aligned");
  return FA_OK;
}

fa_status fa_fwd_varlen(const fa_varlen_params* params, fa_stream_t stream) {
  if (!params) return fail(FA_ERR_INVALID_ARG, "params is null");
  const fa_varlen_params& a = *params;
  fa_status st = check_varlen(a);
  if (st != FA_OK) return st;
  if (a.total_q == 0) return FA_OK;  // nothing to compute
  const size_t need = var_layout(a.B, a.H, a.Hkv, a.total_q, a.d).total;
  if ((st = check_workspace(a.workspace, a.workspace_bytes, need)) != FA_OK) return st;
  DeviceInfo dev;
  if ((st = device_info(&dev)) != FA_OK) return st;
  fa::VarLaunch L;
  std::memset(&L, 0, sizeof L);
  fill_var(&L.p, common_of(a), a.o, a.lse, a.o_token, a.cu_seqlens_q, a.workspace, a.total_k,
           a.timeout_us, dev.status);
  L.p.total_k = a.total_k;
  L.p.cu_k = a.cu_seqlens_k;
  L.sms = dev.sms;
  const bool bf16 = a.dtype == FA_BF16;
  if ((st = make_map3(&L.tmQ, a.q, bf16, a.d, a.H, a.d, a.total_q, a.q_token, L.p.G, L.p.TPT)) !=
          FA_OK ||
      (st = make_map3(&L.tmO, a.o, bf16, a.d, a.H, a.d, a.total_q, a.o_token, L.p.G, L.p.TPT)) !=
          FA_OK)
    return st;
  // without keys no block is loaded; the maps only need a valid address
  const bool any = a.total_k > 0;
  const long long rows = any ? a.total_k : 1;
  if ((st = make_map3(&L.tmK, any ? a.k : a.q, bf16, a.d, a.Hkv, a.d, rows,
                      any ? a.k_token : a.q_token, 1, fa::kVarBN)) != FA_OK)
    return st;
  if ((st = make_map3(&L.tmV, any ? a.v : a.q, bf16, a.d, a.Hkv, a.d, rows,
                      any ? a.v_token : a.q_token, 1, fa::kVarBN)) != FA_OK)
    return st;
  const cudaError_t e = fa::launch_varlen(L, a.d, bf16, reinterpret_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "packed attention launch");
  return FA_OK;
}

size_t fa_paged_varlen_workspace_size(int B, int H, int Hkv, int total_q, int max_q,
                                      int max_pages_per_seq, int page_size, int d) {
  (void)max_pages_per_seq;
  (void)page_size;
  if (B < 1 || Hkv < 1 || H < Hkv || H % Hkv || H / Hkv > 128 || total_q < 0 || max_q < 0 || d < 1)
    return 0;
  return few_rows(max_q, H / Hkv) ? fa::kFewHeadBytes + fa::few_part_floats(d) * sizeof(float)
                                  : var_layout(B, H, Hkv, total_q, d).total;
}

// Both paged calls; x: all zeros for the plain one.
static fa_status paged_varlen(const fa_paged_varlen_params& a, const fa_paged_varlen_extra& x,
                              fa_stream_t stream) {
  const Common c{a.B,         a.H,      a.Hkv,      a.d,    a.total_q, a.scale,
                 a.mask_mode, a.window, a.n_global, a.dtype};
  Common checked = c;
  const bool tree = c.mask_mode == FA_MASK_TREE, q8 = x.k_scales != nullptr;
  if (tree) checked.mask_mode = FA_MASK_NONE;
  if (tree != (x.tree != nullptr))
    return fail(FA_ERR_INVALID_ARG, "mask_mode %d: a tree goes with FA_MASK_TREE", c.mask_mode);
  fa_status st = check_common(checked);
  if (st != FA_OK) return st;
  if (tree && (x.tree_words < 1 || x.tree_words > (1 << 26) || 32LL * x.tree_words < a.max_q ||
               !aligned4(x.tree)))
    return fail(FA_ERR_INVALID_ARG,
                "tree: 4-byte aligned, with 32 * tree_words at least max_q = %d", a.max_q);
  if (q8 != (x.v_scales != nullptr) || !aligned16(x.k_scales) || !aligned16(x.v_scales))
    return fail(FA_ERR_INVALID_ARG, "k_scales and v_scales: both or neither, 16-byte aligned");
  if (a.max_pages_per_seq < 1 || a.num_pages < 1 || a.max_q < 0)
    return fail(FA_ERR_INVALID_ARG, "need max_pages_per_seq, num_pages >= 1 and max_q >= 0");
  if (a.page_size < 16 || a.page_size > 4096 || a.page_size % 16 != 0)
    return fail(FA_ERR_UNSUPPORTED, "page_size %d (a multiple of 16 in [16, 4096])", a.page_size);
  const long long cap = static_cast<long long>(a.page_size) * a.max_pages_per_seq;
  if (cap > (1LL << 30) || static_cast<long long>(a.num_pages) * a.Hkv > (1LL << 31) - 1)
    return fail(FA_ERR_INVALID_ARG, "problem too large");
  // few rows number the 64-key tiles of a sequence's K/V heads in 32 bits, and a CTA's run too
  const bool few = few_rows(a.max_q, a.H / a.Hkv);
  const long long tiles = (cap + 63) / 64 * a.Hkv;
  if (few && (tiles > (1LL << 31) - 1 || tiles * a.B > (1LL << 38)))
    return fail(FA_ERR_INVALID_ARG, "problem too large");
  if (a.total_q == 0) return FA_OK;
  if ((st = check_packed("q", a.q, a.q_token, a.H, a.d)) != FA_OK) return st;
  if ((st = check_packed("o", a.o, a.o_token, a.H, a.d)) != FA_OK) return st;
  if (!a.k_pages || !a.v_pages || !aligned16(a.k_pages) || !aligned16(a.v_pages))
    return fail(FA_ERR_INVALID_ARG, "pools: non-null, 16-byte aligned");
  if (!a.block_table || !a.ctx_lens || !a.cu_seqlens_q || !aligned4(a.block_table) ||
      !aligned4(a.ctx_lens) || !aligned4(a.cu_seqlens_q))
    return fail(FA_ERR_INVALID_ARG,
                "block_table, ctx_lens and cu_seqlens_q: non-null, 4-byte aligned");
  if (!aligned4(a.lse)) return fail(FA_ERR_INVALID_ARG, "lse must be 4-byte aligned");
  const size_t need = fa_paged_varlen_workspace_size(a.B, a.H, a.Hkv, a.total_q, a.max_q,
                                                     a.max_pages_per_seq, a.page_size, a.d);
  if ((st = check_workspace(a.workspace, a.workspace_bytes, need)) != FA_OK) return st;
  DeviceInfo dev;
  if ((st = device_info(&dev)) != FA_OK) return st;
  const bool bf16 = a.dtype == FA_BF16;
  const cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
  // pools as (d, page, num_pages * Hkv); a box is rows of one page, a power of two of them
  const long long planes = static_cast<long long>(a.num_pages) * a.Hkv;
  const long long plane = static_cast<long long>(a.page_size) * a.d;
  const int pow2 = a.page_size & -a.page_size;
  if (few) {
    fa::FewLaunch F;
    std::memset(&F, 0, sizeof F);
    fa::FewParams& p = F.p;
    fill_mask(&p.m, c, a.timeout_us, dev.status);
    p.q = a.q;
    p.o = a.o;
    p.lse = a.lse;
    p.q_token = a.q_token;
    p.o_token = a.o_token;
    p.cu_q = a.cu_seqlens_q;
    p.ctx = a.ctx_lens;
    p.block_table = a.block_table;
    p.B = a.B;
    p.H = a.H;
    p.Hkv = a.Hkv;
    p.G = a.H / a.Hkv;
    p.total_q = a.total_q;
    p.max_q = a.max_q;
    p.page_size = a.page_size;
    p.max_pages = a.max_pages_per_seq;
    p.num_pages = a.num_pages;
    p.box = std::min(q8 ? fa::kFew8Tile : 64, pow2);
    p.heads = static_cast<fa::FewHead*>(a.workspace);
    const bool more = q8 && a.max_q * p.G <= 8;  // CTAs
    p.part = reinterpret_cast<float*>(static_cast<uint8_t*>(a.workspace) +
                                      (more ? fa::kFew8HeadBytes : fa::kFewHeadBytes));
    p.k_scales = x.k_scales;
    p.v_scales = x.v_scales;
    p.tree = x.tree;
    p.tree_words = x.tree_words;
    F.sms = dev.sms;
    if (q8) {
      if ((st = make_map8(&F.tmK, a.k_pages, a.d, a.page_size, planes, p.box)) != FA_OK ||
          (st = make_map8(&F.tmV, a.v_pages, a.d, a.page_size, planes, p.box)) != FA_OK)
        return st;
    } else if ((st = make_map3(&F.tmK, a.k_pages, bf16, a.d, a.page_size, a.d, planes, plane,
                               p.box, 1)) != FA_OK ||
               (st = make_map3(&F.tmV, a.v_pages, bf16, a.d, a.page_size, a.d, planes, plane,
                               p.box, 1)) != FA_OK) {
      return st;
    }
    const cudaError_t e = q8 ? fa::launch_few8(F, a.d, bf16, cs) : fa::launch_few(F, a.d, bf16, cs);
    if (e != cudaSuccess) return cuda_fail(e, "paged packed attention launch");
    return FA_OK;
  }
  fa::VarLaunch L;
  std::memset(&L, 0, sizeof L);
  fill_var(&L.p, c, a.o, a.lse, a.o_token, a.cu_seqlens_q, a.workspace, cap, a.timeout_us,
           dev.status);
  L.p.ctx = a.ctx_lens;
  L.p.block_table = a.block_table;
  L.p.page_size = a.page_size;
  L.p.max_pages = a.max_pages_per_seq;
  L.p.num_pages = a.num_pages;
  L.p.box = std::min(fa::kVarBN, pow2);
  L.p.k_pages = a.k_pages;
  L.p.v_pages = a.v_pages;
  L.p.k_scales = x.k_scales;
  L.p.v_scales = x.v_scales;
  L.p.tree = x.tree;
  L.p.tree_words = x.tree_words;
  L.runs = q8 || tree;
  L.sms = dev.sms;
  if ((st = make_map3(&L.tmQ, a.q, bf16, a.d, a.H, a.d, a.total_q, a.q_token, L.p.G, L.p.TPT)) !=
          FA_OK ||
      (st = make_map3(&L.tmO, a.o, bf16, a.d, a.H, a.d, a.total_q, a.o_token, L.p.G, L.p.TPT)) !=
          FA_OK)
    return st;
  // (the tiles of an 8-bit cache are loaded as they lie there, without a map)
  if (!q8 && ((st = make_map3(&L.tmK, a.k_pages, bf16, a.d, a.page_size, a.d, planes, plane,
                              L.p.box, 1)) != FA_OK ||
              (st = make_map3(&L.tmV, a.v_pages, bf16, a.d, a.page_size, a.d, planes, plane,
                              L.p.box, 1)) != FA_OK))
    return st;
  const cudaError_t e = fa::launch_varlen(L, a.d, bf16, cs);
  if (e != cudaSuccess) return cuda_fail(e, "paged packed attention launch");
  return FA_OK;
}

fa_status fa_fwd_paged_varlen(const fa_paged_varlen_params* params, fa_stream_t stream) {
  if (!params) return fail(FA_ERR_INVALID_ARG, "params is null");
  return paged_varlen(*params, fa_paged_varlen_extra{nullptr, nullptr, nullptr, 0}, stream);
}

fa_status fa_fwd_paged_varlen_ex(const fa_paged_varlen_params* params,
                                 const fa_paged_varlen_extra* extra, fa_stream_t stream) {
  if (!params || !extra) return fail(FA_ERR_INVALID_ARG, "params or extra is null");
  return paged_varlen(*params, *extra, stream);
}

size_t fa_bwd_varlen_workspace_size(int B, int H, int Hkv, int total_q, int total_k, int d) {
  if (B < 1 || Hkv < 1 || H < Hkv || H % Hkv || H / Hkv > 128 || total_q < 0 || total_k < 0 ||
      d < 1)
    return 0;
  return bwd_layout(B, H, Hkv, total_q, total_k, d).total;
}

fa_status fa_bwd_varlen(const fa_varlen_params* params, const fa_varlen_grads* grads,
                        fa_stream_t stream) {
  if (!params || !grads) return fail(FA_ERR_INVALID_ARG, "params or grads is null");
  const fa_varlen_params& a = *params;
  const fa_varlen_grads& g = *grads;
  fa_status st = check_varlen(a);
  if (st != FA_OK) return st;
  if (a.total_q > 0) {
    if (!a.lse) return fail(FA_ERR_INVALID_ARG, "lse must be non-null");
    if ((st = check_packed("dout", g.dout, g.dout_token, a.H, a.d)) != FA_OK) return st;
    if ((st = check_packed("dq", g.dq, g.dq_token, a.H, a.d)) != FA_OK) return st;
  }
  if (a.total_k > 0) {
    if ((st = check_packed("dk", g.dk, g.dk_token, a.Hkv, a.d)) != FA_OK) return st;
    if ((st = check_packed("dv", g.dv, g.dv_token, a.Hkv, a.d)) != FA_OK) return st;
  }
  if (a.total_q == 0 && a.total_k == 0) return FA_OK;
  const BwdLayout B = bwd_layout(a.B, a.H, a.Hkv, a.total_q, a.total_k, a.d);
  if ((st = check_workspace(a.workspace, a.workspace_bytes, B.total)) != FA_OK) return st;
  if (static_cast<long long>(B.max_units) * a.Hkv * B.HS > (1LL << 31) - 1 ||
      static_cast<long long>(a.Hkv) * B.HS > 65535)
    return fail(FA_ERR_INVALID_ARG, "problem too large");
  DeviceInfo dev;
  if ((st = device_info(&dev)) != FA_OK) return st;
  fa::VarBwdLaunch L;
  std::memset(&L, 0, sizeof L);
  fa::VarBwdParams& p = L.p;
  fill_mask(&p.m, common_of(a), a.timeout_us, dev.status);
  p.o = a.o;
  p.dout = g.dout;
  p.lse = a.lse;
  p.dq = g.dq;
  p.dk = g.dk;
  p.dv = g.dv;
  p.o_token = a.o_token;
  p.dout_token = g.dout_token;
  p.dq_token = g.dq_token;
  p.dk_token = g.dk_token;
  p.dv_token = g.dv_token;
  p.cu_q = a.cu_seqlens_q;
  p.cu_k = a.cu_seqlens_k;
  p.scale = a.scale;
  p.B = a.B;
  p.H = a.H;
  p.Hkv = a.Hkv;
  p.G = a.H / a.Hkv;
  p.GS = B.GS;
  p.HS = B.HS;
  p.TPH = B.TPH;
  p.total_q = a.total_q;
  p.total_k = a.total_k;
  p.slots = B.slots;
  p.max_units = B.max_units;
  while (((a.total_q / B.TPH + 1) >> p.cost_shift) >= 1024) ++p.cost_shift;
  uint8_t* ws = static_cast<uint8_t*>(a.workspace);
  p.n_units = reinterpret_cast<int32_t*>(ws);
  p.units = reinterpret_cast<fa::VarBwdUnit*>(ws + B.units);
  p.seq_slot = reinterpret_cast<int32_t*>(ws + B.seq_slot);
  p.stats = reinterpret_cast<float*>(ws + B.stats);
  p.dqacc = reinterpret_cast<float*>(ws + B.dqacc);
  p.part = reinterpret_cast<float*>(ws + B.part);
  const bool bf16 = a.dtype == FA_BF16;
  // a side without rows is never loaded; its maps only need a valid address
  const bool nq = a.total_q > 0, nk = a.total_k > 0;
  const void* q = nq ? a.q : a.k;
  const void* dout = nq ? g.dout : a.k;
  const int qh = nq ? a.H : a.Hkv, kh = nk ? a.Hkv : a.H;
  const int gs = std::min(B.GS, qh);
  const long long qn = nq ? a.total_q : 1, kn = nk ? a.total_k : 1;
  const long long qt = nq ? a.q_token : a.k_token, ot = nq ? g.dout_token : a.k_token;
  const long long kt = nk ? a.k_token : a.q_token, vt = nk ? a.v_token : a.q_token;
  if ((st = make_map3(&L.tmQ, q, bf16, a.d, qh, a.d, qn, qt, gs, B.TPH)) != FA_OK) return st;
  if ((st = make_map3(&L.tmdO, dout, bf16, a.d, qh, a.d, qn, ot, gs, B.TPH)) != FA_OK) return st;
  if ((st = make_map3(&L.tmK, nk ? a.k : a.q, bf16, a.d, kh, a.d, kn, kt, 1, 64)) != FA_OK)
    return st;
  if ((st = make_map3(&L.tmV, nk ? a.v : a.q, bf16, a.d, kh, a.d, kn, vt, 1, 64)) != FA_OK)
    return st;
  const cudaError_t e = fa::launch_bwd_varlen(L, a.d, bf16, reinterpret_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "packed backward launch");
  return FA_OK;
}

}  // extern "C"
