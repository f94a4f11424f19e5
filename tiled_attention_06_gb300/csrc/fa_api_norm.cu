// The C ABI of the calls between a projection and a paged cache (include/fa.h): norms with rotary
// positions and their gradient, the form that writes the cache, and reading an 8-bit cache back.
// Every check runs on the host before anything is launched.
#include <cuda.h>
#include <cuda_runtime.h>

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
using fa::host::fail;

bool aligned8(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 7u) == 0; }
size_t elem_size(int dtype) { return dtype == FA_F32 ? 4 : 2; }

// Rows of heads, element e of head h of token t at t * token + h * head + e.
struct Rows {
  const char* name;
  const void* ptr;
  int64_t token, head;
  bool written;
};

fa_status check_rows(const Rows& r, int64_t T, int H, int d, size_t es) {
  if (!r.ptr) return fail(FA_ERR_INVALID_ARG, "%s must be non-null", r.name);
  if (reinterpret_cast<uintptr_t>(r.ptr) % es)
    return fail(FA_ERR_INVALID_ARG, "%s must be aligned to its elements", r.name);
  if (r.head < d || r.token < 0 || r.token > (1LL << 38) || r.head > (1LL << 38))
    return fail(FA_ERR_INVALID_ARG,
                "%s: heads must be at least d elements apart, tokens not negative", r.name);
  const int64_t row = static_cast<int64_t>(H - 1) * r.head + d;
  if (r.written && T > 1 && r.token < row &&
      !(r.head >= (T - 1) * r.token + d && r.token >= d))
    return fail(FA_ERR_INVALID_ARG, "the rows of %s overlap", r.name);
  return FA_OK;
}
fa_status check_in_place(const Rows& in, const Rows& out) {
  if (in.ptr == out.ptr && (in.token != out.token || in.head != out.head))
    return fail(FA_ERR_INVALID_ARG, "in place, %s and %s have the same steps", in.name, out.name);
  return FA_OK;
}
bool wide(const Rows& r, size_t es) {
  const int64_t v = 16 / static_cast<int64_t>(es);
  return aligned16(r.ptr) && r.token % v == 0 && r.head % v == 0;
}

// What the calls with a norm and a rotation have in common.
struct Turn {
  int d, rot_dim, axes, style, norm, weight_dtype, dtype;
  float amplitude, eps;
  const int32_t* positions;
  const int32_t* pair_axis;
  const double* freqs;
  const void* q_weight;
  const void* k_weight;
};

fa_status check_turn(const Turn& t) {
  if (t.dtype != FA_F16 && t.dtype != FA_BF16 && t.dtype != FA_F32)
    return fail(FA_ERR_UNSUPPORTED, "dtype %d", t.dtype);
  if (t.d < 2 || t.d > 512) return fail(FA_ERR_INVALID_ARG, "head dim %d (in [2, 512])", t.d);
  if (t.d % 2) return fail(FA_ERR_UNSUPPORTED, "head dim %d (even)", t.d);
  if (t.rot_dim < 2 || t.rot_dim > t.d || t.rot_dim % 2)
    return fail(FA_ERR_INVALID_ARG, "rot_dim %d (even, in [2, d])", t.rot_dim);
  if (t.axes < 1 || t.axes > FA_MAX_AXES)
    return fail(FA_ERR_INVALID_ARG, "%d axes (1 to %d)", t.axes, FA_MAX_AXES);
  if (t.style != FA_ROPE_HALF && t.style != FA_ROPE_PAIRS)
    return fail(FA_ERR_INVALID_ARG, "style %d", t.style);
  if (!std::isfinite(t.amplitude)) return fail(FA_ERR_INVALID_ARG, "amplitude must be finite");
  if (t.norm != FA_NORM_NONE && t.norm != FA_NORM_RMS)
    return fail(FA_ERR_INVALID_ARG, "norm %d", t.norm);
  if (t.norm == FA_NORM_RMS) {
    if (!(t.eps >= 0) || !std::isfinite(t.eps))
      return fail(FA_ERR_INVALID_ARG, "eps must be finite and not negative");
    if (t.weight_dtype != FA_F32 && t.weight_dtype != t.dtype)
      return fail(FA_ERR_INVALID_ARG, "weight_dtype %d (FA_F32 or dtype)", t.weight_dtype);
    const size_t es = elem_size(t.weight_dtype);
    if (reinterpret_cast<uintptr_t>(t.q_weight) % es || reinterpret_cast<uintptr_t>(t.k_weight) % es)
      return fail(FA_ERR_INVALID_ARG, "weights must be aligned to their elements");
  }
  return FA_OK;
}
fa_status check_turn_arrays(const Turn& t) {
  if (!t.freqs || !aligned8(t.freqs))
    return fail(FA_ERR_INVALID_ARG, "freqs: non-null, 8-byte aligned");
  if (!aligned4(t.positions) || !aligned4(t.pair_axis))
    return fail(FA_ERR_INVALID_ARG, "positions and pair_axis must be 4-byte aligned");
  if (t.axes > 1 && !t.pair_axis)
    return fail(FA_ERR_INVALID_ARG, "several axes need a pair_axis");
  return FA_OK;
}
void fill_turn(fa::NormRopeParams* p, const Turn& t) {
  p->d = t.d;
  p->rot = t.rot_dim;
  p->axes = t.axes;
  p->norm = t.norm == FA_NORM_RMS;
  p->w_f32 = t.weight_dtype == FA_F32;
  p->amplitude = t.amplitude;
  p->eps = t.eps;
  p->pos = t.positions;
  p->pair_axis = t.pair_axis;
  p->freqs = t.freqs;
  p->q_weight = t.norm == FA_NORM_RMS ? t.q_weight : nullptr;
  p->k_weight = t.norm == FA_NORM_RMS ? t.k_weight : nullptr;
}
// (without key heads k_weight is ignored; lanes without a head would read its first element)
Turn turn_of(const fa_norm_rope_params& a) {
  return Turn{a.d,       a.rot_dim,   a.axes,  a.style,    a.norm, a.weight_dtype, a.dtype, a.amplitude, a.eps,
              a.positions, a.pair_axis, a.freqs, a.q_weight, a.Hkv ? a.k_weight : nullptr};
}

fa_status check_sizes(const fa_norm_rope_params& a) {
  if (a.T < 0 || a.H < 1 || a.Hkv < 0)
    return fail(FA_ERR_INVALID_ARG, "need T, Hkv >= 0 and H >= 1");
  if (a.T > (1LL << 33) || a.H > (1 << 16) || a.Hkv > (1 << 16) ||
      static_cast<int64_t>(a.H) * a.d > (1LL << 28))
    return fail(FA_ERR_INVALID_ARG, "problem too large");
  return FA_OK;
}

fa_status check_paging(int B, int Hkv, int d, int page_size, int max_pages, int num_pages) {
  if (B < 1 || Hkv < 1 || max_pages < 1 || num_pages < 1)
    return fail(FA_ERR_INVALID_ARG, "need B, Hkv, max_pages_per_seq and num_pages >= 1");
  if (d != 64 && d != 128) return fail(FA_ERR_UNSUPPORTED, "head dim %d (supported: 64, 128)", d);
  if (page_size < 16 || page_size > 4096 || page_size % 16 != 0)
    return fail(FA_ERR_UNSUPPORTED, "page_size %d (a multiple of 16 in [16, 4096])", page_size);
  if (Hkv > (1 << 16) || B > (1 << 24) ||
      static_cast<long long>(page_size) * max_pages > (1LL << 30))
    return fail(FA_ERR_INVALID_ARG, "problem too large");
  return FA_OK;
}

}  // namespace

extern "C" {

fa_status fa_rope_axes(int32_t* pair_axis, int rot_dim, const int32_t* sections, int axes,
                       int interleaved) {
  if (!pair_axis || !sections)
    return fail(FA_ERR_INVALID_ARG, "pair_axis and sections must be non-null");
  if (rot_dim < 2 || rot_dim > 512 || rot_dim % 2)
    return fail(FA_ERR_INVALID_ARG, "rot_dim %d (even, in [2, 512])", rot_dim);
  if (axes < 1 || axes > FA_MAX_AXES)
    return fail(FA_ERR_INVALID_ARG, "%d axes (1 to %d)", axes, FA_MAX_AXES);
  long long sum = 0;
  int left[FA_MAX_AXES] = {0, 0, 0, 0};
  for (int a = 0; a < axes; ++a) {
    if (sections[a] < 0) return fail(FA_ERR_INVALID_ARG, "section %d is negative", a);
    left[a] = sections[a];
    sum += sections[a];
  }
  if (sum != rot_dim / 2)
    return fail(FA_ERR_INVALID_ARG, "sections add up to %lld pairs, not rot_dim / 2 = %d", sum,
                rot_dim / 2);
  for (int i = 0, a = 0; i < rot_dim / 2; ++i) {
    while (left[a] == 0) a = (a + 1) % axes;  // some axis has pairs left
    pair_axis[i] = a;
    --left[a];
    if (interleaved) a = (a + 1) % axes;
  }
  return FA_OK;
}

fa_status fa_norm_rope(const fa_norm_rope_params* params, fa_stream_t stream) {
  if (!params) return fail(FA_ERR_INVALID_ARG, "params is null");
  const fa_norm_rope_params& a = *params;
  const Turn t = turn_of(a);
  fa_status st = check_turn(t);
  if (st != FA_OK || (st = check_sizes(a)) != FA_OK) return st;
  if (a.T == 0) return FA_OK;
  if ((st = check_turn_arrays(t)) != FA_OK) return st;
  if (!a.positions) return fail(FA_ERR_INVALID_ARG, "positions must be non-null");
  const size_t es = elem_size(a.dtype);
  const Rows rows[4] = {{"q", a.q, a.q_token, a.q_head, false},
                        {"q_out", a.q_out, a.q_out_token, a.q_out_head, true},
                        {"k", a.k, a.k_token, a.k_head, false},
                        {"k_out", a.k_out, a.k_out_token, a.k_out_head, true}};
  bool vec = true;
  for (int i = 0; i < (a.Hkv ? 4 : 2); ++i) {
    if ((st = check_rows(rows[i], a.T, i < 2 ? a.H : a.Hkv, a.d, es)) != FA_OK) return st;
    if (i % 2 && (st = check_in_place(rows[i - 1], rows[i])) != FA_OK) return st;
    vec = vec && wide(rows[i], es);
  }
  DeviceInfo dev;
  if ((st = device_info(&dev)) != FA_OK) return st;
  fa::NormRopeParams p;
  std::memset(&p, 0, sizeof p);
  fill_turn(&p, t);
  p.q = a.q;
  p.k = a.k;
  p.q_out = a.q_out;
  p.k_out = a.k_out;
  p.q_token = a.q_token;
  p.q_head = a.q_head;
  p.k_token = a.k_token;
  p.k_head = a.k_head;
  p.q_out_token = a.q_out_token;
  p.q_out_head = a.q_out_head;
  p.k_out_token = a.k_out_token;
  p.k_out_head = a.k_out_head;
  p.T = a.T;
  p.H = a.H;
  p.Hkv = a.Hkv;
  p.status = dev.status;
  const cudaError_t e = fa::launch_norm_rope(p, a.dtype, a.style == FA_ROPE_HALF, vec, dev.sms,
                                             reinterpret_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "norm rope launch");
  return FA_OK;
}

size_t fa_norm_rope_bwd_workspace_size(int H, int Hkv, int d) {
  if (H < 1 || Hkv < 0 || H > (1 << 16) || Hkv > (1 << 16) || d < 2 || d > 512) return 0;
  return static_cast<size_t>(fa::norm_parts(H + Hkv)) * 2 * d * sizeof(float);
}

fa_status fa_norm_rope_bwd(const fa_norm_rope_params* params, const fa_norm_rope_grads* grads,
                           fa_stream_t stream) {
  if (!params || !grads) return fail(FA_ERR_INVALID_ARG, "params or grads is null");
  const fa_norm_rope_params& a = *params;
  const fa_norm_rope_grads& g = *grads;
  const Turn t = turn_of(a);
  fa_status st = check_turn(t);
  if (st != FA_OK || (st = check_sizes(a)) != FA_OK) return st;
  const bool norm = a.norm == FA_NORM_RMS;
  if (!norm && (g.dq_weight || g.dk_weight))
    return fail(FA_ERR_INVALID_ARG, "without a norm there is no gradient of a weight");
  if (!aligned4(g.dq_weight) || !aligned4(g.dk_weight))
    return fail(FA_ERR_INVALID_ARG, "the weights' gradients must be 4-byte aligned");
  const bool want = g.dq_weight || (g.dk_weight && a.Hkv);
  const cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
  if (a.T == 0 || !a.Hkv) {  // sums over nothing
    for (float* w : {a.T == 0 ? g.dq_weight : nullptr, g.dk_weight}) {
      if (!w) continue;
      const cudaError_t e = cudaMemsetAsync(w, 0, sizeof(float) * a.d, cs);
      if (e != cudaSuccess) return cuda_fail(e, "norm rope backward");
    }
    if (a.T == 0) return FA_OK;
  }
  if ((st = check_turn_arrays(t)) != FA_OK) return st;
  if (!a.positions) return fail(FA_ERR_INVALID_ARG, "positions must be non-null");
  const size_t es = elem_size(a.dtype);
  const Rows rows[6] = {{"dq_out", g.dq_out, g.dq_out_token, g.dq_out_head, false},
                        {"dq", g.dq, g.dq_token, g.dq_head, true},
                        {"q", a.q, a.q_token, a.q_head, false},
                        {"dk_out", g.dk_out, g.dk_out_token, g.dk_out_head, false},
                        {"dk", g.dk, g.dk_token, g.dk_head, true},
                        {"k", a.k, a.k_token, a.k_head, false}};
  bool vec = true;
  for (int i = 0; i < (a.Hkv ? 6 : 3); ++i) {
    if (i % 3 == 2 && !norm) continue;  // the input is not read
    if ((st = check_rows(rows[i], a.T, i < 3 ? a.H : a.Hkv, a.d, es)) != FA_OK) return st;
    if (i % 3 == 1 && (st = check_in_place(rows[i - 1], rows[i])) != FA_OK) return st;
    vec = vec && wide(rows[i], es);
  }
  if (want) {
    const size_t need = fa_norm_rope_bwd_workspace_size(a.H, a.Hkv, a.d);
    if (!g.workspace || !aligned16(g.workspace))
      return fail(FA_ERR_INVALID_ARG, "a 16-byte aligned workspace is needed");
    if (g.workspace_bytes < need)
      return fail(FA_ERR_INVALID_ARG, "workspace has %zu bytes, needs %zu", g.workspace_bytes, need);
  }
  DeviceInfo dev;
  if ((st = device_info(&dev)) != FA_OK) return st;
  fa::NormRopeParams p;
  std::memset(&p, 0, sizeof p);
  fill_turn(&p, t);
  p.T = a.T;
  p.H = a.H;
  p.Hkv = a.Hkv;
  p.inverse = 1;
  p.status = dev.status;
  p.q_out = g.dq;
  p.k_out = g.dk;
  p.q_out_token = g.dq_token;
  p.q_out_head = g.dq_head;
  p.k_out_token = g.dk_token;
  p.k_out_head = g.dk_head;
  cudaError_t e;
  if (!norm) {  // the rotation's transpose alone
    p.q = g.dq_out;
    p.k = g.dk_out;
    p.q_token = g.dq_out_token;
    p.q_head = g.dq_out_head;
    p.k_token = g.dk_out_token;
    p.k_head = g.dk_out_head;
    e = fa::launch_norm_rope(p, a.dtype, a.style == FA_ROPE_HALF, vec, dev.sms, cs);
  } else {
    p.q = a.q;
    p.k = a.k;
    p.q_token = a.q_token;
    p.q_head = a.q_head;
    p.k_token = a.k_token;
    p.k_head = a.k_head;
    p.dyq = g.dq_out;
    p.dyk = g.dk_out;
    p.dyq_token = g.dq_out_token;
    p.dyq_head = g.dq_out_head;
    p.dyk_token = g.dk_out_token;
    p.dyk_head = g.dk_out_head;
    p.part = want ? static_cast<float*>(g.workspace) : nullptr;
    p.dq_weight = g.dq_weight;
    p.dk_weight = a.Hkv ? g.dk_weight : nullptr;
    e = fa::launch_norm_rope_bwd(p, a.dtype, a.style == FA_ROPE_HALF, vec, dev.sms, cs);
  }
  if (e != cudaSuccess) return cuda_fail(e, "norm rope backward launch");
  return FA_OK;
}

fa_status fa_norm_rope_append(const fa_norm_rope_append_params* params, fa_stream_t stream) {
  if (!params) return fail(FA_ERR_INVALID_ARG, "params is null");
  const fa_norm_rope_append_params& a = *params;
  const Turn t{a.d,   a.rot_dim,   a.axes,      a.style, a.norm,     a.weight_dtype, a.dtype, a.amplitude,
               a.eps, a.positions, a.pair_axis, a.freqs, a.q_weight, a.k_weight};
  fa_status st = check_turn(t);
  if (st != FA_OK) return st;
  if (a.dtype == FA_F32) return fail(FA_ERR_UNSUPPORTED, "dtype %d", a.dtype);
  if (a.T < 0 || a.H < 1) return fail(FA_ERR_INVALID_ARG, "need H >= 1 and T >= 0");
  if ((st = check_paging(a.B, a.Hkv, a.d, a.page_size, a.max_pages_per_seq, a.num_pages)) != FA_OK)
    return st;
  if (a.H > (1 << 16) || a.T > (1 << 30)) return fail(FA_ERR_INVALID_ARG, "problem too large");
  if ((a.k_scales == nullptr) != (a.v_scales == nullptr))
    return fail(FA_ERR_INVALID_ARG, "k_scales and v_scales: both or neither");
  if (a.T == 0) return FA_OK;
  if ((st = check_turn_arrays(t)) != FA_OK) return st;
  if (!a.positions && a.axes != 1)
    return fail(FA_ERR_INVALID_ARG, "several axes need positions");
  if ((st = check_packed("q", a.q, a.q_token, a.H, a.d)) != FA_OK) return st;
  if ((st = check_packed("q_out", a.q_out, a.q_out_token, a.H, a.d)) != FA_OK) return st;
  if ((st = check_packed("k", a.k, a.k_token, a.Hkv, a.d)) != FA_OK) return st;
  if ((st = check_packed("v", a.v, a.v_token, a.Hkv, a.d)) != FA_OK) return st;
  if (a.q == a.q_out && a.q_token != a.q_out_token)
    return fail(FA_ERR_INVALID_ARG, "in place, q and q_out have the same step");
  if (!a.k_pages || !a.v_pages || !aligned16(a.k_pages) || !aligned16(a.v_pages))
    return fail(FA_ERR_INVALID_ARG, "pools: non-null, 16-byte aligned");
  if (!a.block_table || !a.ctx_lens || !a.cu_seqlens || !aligned4(a.block_table) ||
      !aligned4(a.ctx_lens) || !aligned4(a.cu_seqlens))
    return fail(FA_ERR_INVALID_ARG,
                "block_table, ctx_lens and cu_seqlens: non-null, 4-byte aligned");
  DeviceInfo dev;
  if ((st = device_info(&dev)) != FA_OK) return st;
  fa::NormRopeParams p;
  std::memset(&p, 0, sizeof p);
  fill_turn(&p, t);
  p.q = a.q;
  p.k = a.k;
  p.v = a.v;
  p.q_out = a.q_out;
  p.q_token = a.q_token;
  p.k_token = a.k_token;
  p.v_token = a.v_token;
  p.q_out_token = a.q_out_token;
  p.q_head = p.k_head = p.q_out_head = a.d;
  p.T = a.T;
  p.H = a.H;
  p.Hkv = a.Hkv;
  p.k_pages = a.k_pages;
  p.v_pages = a.v_pages;
  p.k_scales = a.k_scales;
  p.v_scales = a.v_scales;
  p.cu = a.cu_seqlens;
  p.ctx = a.ctx_lens;
  p.block_table = a.block_table;
  p.B = a.B;
  p.page_size = a.page_size;
  p.max_pages = a.max_pages_per_seq;
  p.num_pages = a.num_pages;
  p.status = dev.status;
  const cudaError_t e =
      fa::launch_norm_rope_append(p, a.dtype, a.style == FA_ROPE_HALF, true, dev.sms,
                                  reinterpret_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "norm rope append launch");
  return FA_OK;
}

fa_status fa_kv_read(const fa_kv_read_params* params, fa_stream_t stream) {
  if (!params) return fail(FA_ERR_INVALID_ARG, "params is null");
  const fa_kv_read_params& a = *params;
  if (a.dtype != FA_F16 && a.dtype != FA_BF16) return fail(FA_ERR_UNSUPPORTED, "dtype %d", a.dtype);
  if (a.T < 0 || a.T > (1 << 30)) return fail(FA_ERR_INVALID_ARG, "T %d", a.T);
  fa_status st = check_paging(a.B, a.Hkv, a.d, a.page_size, a.max_pages_per_seq, a.num_pages);
  if (st != FA_OK) return st;
  if (a.T == 0) return FA_OK;
  if ((st = check_packed("k", a.k, a.k_token, a.Hkv, a.d)) != FA_OK) return st;
  if ((st = check_packed("v", a.v, a.v_token, a.Hkv, a.d)) != FA_OK) return st;
  if (!a.k_pages || !a.v_pages || !aligned16(a.k_pages) || !aligned16(a.v_pages))
    return fail(FA_ERR_INVALID_ARG, "pools: non-null, 16-byte aligned");
  if (!a.k_scales || !a.v_scales)
    return fail(FA_ERR_INVALID_ARG, "k_scales and v_scales must be non-null");
  if (!a.block_table || !a.starts || !a.cu_seqlens || !aligned4(a.block_table) ||
      !aligned4(a.starts) || !aligned4(a.cu_seqlens))
    return fail(FA_ERR_INVALID_ARG, "block_table, starts and cu_seqlens: non-null, 4-byte aligned");
  DeviceInfo dev;
  if ((st = device_info(&dev)) != FA_OK) return st;
  const fa::KvReadParams p{a.k_pages, a.v_pages, a.k_scales, a.v_scales,  a.block_table,
                           a.starts,  a.cu_seqlens, a.k,     a.v,         a.k_token,
                           a.v_token, a.T,       a.B,        a.Hkv,       a.d,
                           a.page_size, a.max_pages_per_seq, a.num_pages, dev.status};
  const cudaError_t e = fa::launch_kv_read(p, a.dtype == FA_BF16, dev.sms,
                                           reinterpret_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "cache read launch");
  return FA_OK;
}

}  // extern "C"
