"""FlashAttention forward (prefill + paged decode) for one NVIDIA GB300 (sm_103a).

A thin ctypes binding over the C-ABI library ``libfa.so`` (declared in
``include/fa.h``). The functions keep the C names; they only marshal torch
tensors into pointers, sizes and the current CUDA stream. Every step of the
computation runs in the library's CUDA kernels: there is no fallback, and a
missing library raises ``FaError``.
"""
import ctypes
import operator
import os
import struct

import torch

__all__ = [
    "FaError", "lib", "fa_fwd", "fa_fwd_ex", "fa_decode_paged", "fa_decode_paged_ex",
    "fa_decode_paged_noalloc", "fa_merge_partials", "fa_fwd_paged", "fa_fwd_paged_host_lens",
    "fa_kv_append",
    "fa_decode_workspace_size", "fa_decode_default_pages_per_split",
    "fa_get_device_status",
    "fa_selftest_timeout", "fa_last_error_string", "fa_version", "fa_fwd_block_m",
    "fa_fwd_default_block_m", "fa_bwd", "fa_bwd_block_sparse", "fa_bwd_workspace_size", "fa_fwd_workspace_size",
    "fa_rope_freqs", "fa_rope", "fa_rope_append", "fa_fwd_varlen", "fa_bwd_varlen",
    "fa_fwd_paged_varlen", "fa_varlen_workspace_size", "fa_bwd_varlen_workspace_size",
    "fa_paged_varlen_workspace_size", "FA_ROPE_HALF", "FA_ROPE_PAIRS", "FA_ROPE_PLAIN",
    "FA_ROPE_LINEAR", "FA_ROPE_BASE", "FA_ROPE_BY_PARTS",
    "FA_OK", "FA_ERR_INVALID_ARG", "FA_ERR_UNSUPPORTED", "FA_ERR_CUDA", "FA_ERR_TIMEOUT",
    "FA_ERR_BAD_PAGE", "FA_F16", "FA_BF16", "FA_F32", "FA_MASK_NONE", "FA_MASK_CAUSAL",
    "FA_MASK_CAUSAL_WINDOW", "FA_MASK_BAND", "FA_MASK_PREFIX_LM", "FA_MASK_BLOCK_SPARSE",
    "FA_LAYOUT_BLOCK",
]

FA_OK, FA_ERR_INVALID_ARG, FA_ERR_UNSUPPORTED, FA_ERR_CUDA, FA_ERR_TIMEOUT, FA_ERR_BAD_PAGE = range(6)
FA_F16, FA_BF16, FA_F32 = 0, 1, 2
FA_MASK_NONE, FA_MASK_CAUSAL, FA_MASK_CAUSAL_WINDOW, FA_MASK_BAND, FA_MASK_PREFIX_LM = 0, 1, 2, 3, 4
FA_MASK_BLOCK_SPARSE = 5
FA_LAYOUT_BLOCK = 128
FA_ROPE_HALF, FA_ROPE_PAIRS = 0, 1
FA_ROPE_PLAIN, FA_ROPE_LINEAR, FA_ROPE_BASE, FA_ROPE_BY_PARTS = 0, 1, 2, 3

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libfa.so")

_vp = ctypes.c_void_p
_i = ctypes.c_int
_f = ctypes.c_float
_u32 = ctypes.c_uint32
_sz = ctypes.c_size_t
_i64 = ctypes.c_int64


class FaError(RuntimeError):
    def __init__(self, status, msg):
        super().__init__(f"fa status {status}: {msg}")
        self.status = status


class FwdParams(ctypes.Structure):
    _fields_ = [("q", _vp), ("k", _vp), ("v", _vp), ("o", _vp), ("lse", _vp),
                ("B", _i), ("H", _i), ("Sq", _i), ("Sk", _i), ("d", _i), ("scale", _f),
                ("mask_mode", _i), ("window", _i), ("n_global", _i), ("dtype", _i),
                ("block_n", _i), ("block_m", _i), ("num_ctas", _i), ("group_heads", _i),
                ("timeout_us", _u32),
                ("trace", _vp), ("block_layout", _vp), ("workspace", _vp),
                ("workspace_bytes", _sz), ("rescale_count", _vp), ("block_layout_host", _vp)]


class DecodeParams(ctypes.Structure):
    _fields_ = [("q", _vp), ("k_pages", _vp), ("v_pages", _vp), ("block_table", _vp),
                ("ctx_lens", _vp), ("o", _vp), ("lse", _vp), ("B", _i), ("H", _i), ("d", _i),
                ("page_size", _i), ("max_pages_per_seq", _i), ("num_pages", _i), ("scale", _f),
                ("dtype", _i), ("workspace", _vp), ("workspace_bytes", _sz),
                ("pages_per_split", _i), ("trace_pages", _vp), ("trace_splits", _vp)]


class RopeAppendParams(ctypes.Structure):
    _fields_ = [("q", _vp), ("k", _vp), ("v", _vp), ("q_out", _vp), ("k_pages", _vp),
                ("v_pages", _vp), ("block_table", _vp), ("ctx_lens", _vp), ("cu_seqlens", _vp),
                ("freqs", _vp), ("q_token", _i64), ("k_token", _i64), ("v_token", _i64),
                ("q_out_token", _i64), ("T", _i), ("B", _i), ("H", _i), ("Hkv", _i), ("d", _i),
                ("rot_dim", _i), ("page_size", _i), ("max_pages_per_seq", _i), ("num_pages", _i),
                ("style", _i), ("amplitude", _f), ("dtype", _i)]


class VarlenParams(ctypes.Structure):
    _fields_ = [("q", _vp), ("k", _vp), ("v", _vp), ("o", _vp), ("lse", _vp),
                ("q_token", _i64), ("k_token", _i64), ("v_token", _i64), ("o_token", _i64),
                ("cu_seqlens_q", _vp), ("cu_seqlens_k", _vp), ("B", _i), ("H", _i), ("Hkv", _i),
                ("d", _i), ("total_q", _i), ("total_k", _i), ("scale", _f), ("mask_mode", _i),
                ("window", _i), ("n_global", _i), ("dtype", _i), ("workspace", _vp),
                ("workspace_bytes", _sz), ("timeout_us", _u32)]


class VarlenGrads(ctypes.Structure):
    _fields_ = [("dout", _vp), ("dq", _vp), ("dk", _vp), ("dv", _vp), ("dout_token", _i64),
                ("dq_token", _i64), ("dk_token", _i64), ("dv_token", _i64)]


class PagedVarlenParams(ctypes.Structure):
    _fields_ = [("q", _vp), ("k_pages", _vp), ("v_pages", _vp), ("block_table", _vp),
                ("ctx_lens", _vp), ("cu_seqlens_q", _vp), ("o", _vp), ("lse", _vp),
                ("q_token", _i64), ("o_token", _i64), ("B", _i), ("H", _i), ("Hkv", _i),
                ("d", _i), ("total_q", _i), ("max_q", _i), ("page_size", _i),
                ("max_pages_per_seq", _i), ("num_pages", _i), ("scale", _f), ("mask_mode", _i),
                ("window", _i), ("n_global", _i), ("dtype", _i), ("workspace", _vp),
                ("workspace_bytes", _sz), ("timeout_us", _u32)]


_lib = None


def lib():
    """The loaded libfa.so (raises FaError when it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise FaError(FA_ERR_CUDA, f"{LIB_PATH} is missing: build it with "
                          "tiled_attention_06_gb300.build.build()")
        L = ctypes.CDLL(LIB_PATH)
        L.fa_fwd.restype = _i
        L.fa_fwd.argtypes = [_vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _f, _i, _i, _i, _i, _vp]
        L.fa_fwd_ex.restype = _i
        L.fa_fwd_ex.argtypes = [ctypes.POINTER(FwdParams), _vp]
        L.fa_fwd_block_m.restype = _i
        L.fa_fwd_block_m.argtypes = []
        L.fa_fwd_default_block_m.restype = _i
        L.fa_fwd_default_block_m.argtypes = [_i]
        L.fa_fwd_workspace_size.restype = _sz
        L.fa_fwd_workspace_size.argtypes = [_i] * 6
        L.fa_bwd_workspace_size.restype = _sz
        L.fa_bwd_workspace_size.argtypes = [_i, _i, _i]
        L.fa_bwd.restype = _i
        L.fa_bwd.argtypes = [_vp] * 10 + [_sz] + [_i] * 5 + [_f] + [_i] * 4 + [_vp]
        L.fa_bwd_block_sparse.restype = _i
        L.fa_bwd_block_sparse.argtypes = [_vp] * 10 + [_sz] + [_i] * 5 + [_f, _vp, _i, _vp]
        L.fa_decode_paged.restype = _i
        L.fa_decode_paged.argtypes = [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _i,
                                      _f, _i, _vp, _sz, _vp]
        L.fa_decode_paged_ex.restype = _i
        L.fa_decode_paged_ex.argtypes = [ctypes.POINTER(DecodeParams), _vp]
        L.fa_decode_paged_noalloc.restype = _i
        L.fa_decode_paged_noalloc.argtypes = [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i,
                                              _i, _i, _f, _i, _vp]
        L.fa_fwd_paged.restype = _i
        L.fa_fwd_paged.argtypes = [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _i, _i,
                                   _f, _i, _i, _i, _i, _vp]
        L.fa_fwd_paged_host_lens.restype = _i
        L.fa_fwd_paged_host_lens.argtypes = [_vp] * 8 + [_i] * 7 + [_f] + [_i] * 4 + [_vp]
        L.fa_kv_append.restype = _i
        L.fa_kv_append.argtypes = [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _i, _i,
                                   _i, _vp]
        L.fa_merge_partials.restype = _i
        L.fa_merge_partials.argtypes = [_vp, _vp, _vp, _vp, _vp, _vp, ctypes.c_int64, _i, _i, _vp]
        L.fa_decode_workspace_size.restype = _sz
        L.fa_decode_workspace_size.argtypes = [_i, _i, _i, _i, _i]
        L.fa_decode_default_pages_per_split.restype = _i
        L.fa_decode_default_pages_per_split.argtypes = [_i, _i, _i]
        L.fa_get_device_status.restype = _i
        L.fa_get_device_status.argtypes = [_vp]
        L.fa_selftest_timeout.restype = _i
        L.fa_selftest_timeout.argtypes = [_u32, _vp]
        L.fa_last_error_string.restype = ctypes.c_char_p
        L.fa_last_error_string.argtypes = []
        L.fa_version.restype = _i
        L.fa_version.argtypes = []
        L.fa_rope_freqs.restype = _i
        L.fa_rope_freqs.argtypes = [ctypes.POINTER(ctypes.c_double), ctypes.POINTER(_f), _i,
                                    ctypes.c_double, _i, ctypes.c_double, _i, ctypes.c_double,
                                    ctypes.c_double]
        L.fa_rope.restype = _i
        L.fa_rope.argtypes = [_vp] * 4 + [_i64, _i, _i, _i] + [_i64] * 4 + [_i, _f, _i, _i, _vp]
        for name, n in (("fa_rope_append", 1), ("fa_fwd_varlen", 1), ("fa_bwd_varlen", 2),
                        ("fa_fwd_paged_varlen", 1)):  # pointers to their parameter structs
            getattr(L, name).restype = _i
            getattr(L, name).argtypes = [_vp] * n + [_vp]
        for name, n in (("fa_varlen_workspace_size", 6), ("fa_bwd_varlen_workspace_size", 6),
                        ("fa_paged_varlen_workspace_size", 8)):
            getattr(L, name).restype = _sz
            getattr(L, name).argtypes = [_i] * n
        _lib = L
    return _lib


def _check(status):
    if status != FA_OK:
        raise FaError(status, fa_last_error_string())


# The current stream's handle without building a Stream object (2.9 us a call); the public way
# where this torch has no such function.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(stream):
    if stream is None:
        if _raw_stream is not None:
            return _raw_stream(torch.cuda.current_device())
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, torch.cuda.Stream):
        return stream.cuda_stream
    return int(stream)


def _ptr(t):
    return None if t is None else t.data_ptr()


def _dtype_code(t):
    if t.dtype == torch.float16:
        return FA_F16
    if t.dtype == torch.bfloat16:
        return FA_BF16
    if t.dtype == torch.float32:  # fa_fwd / fa_fwd_ex only; the other calls refuse it
        return FA_F32
    raise FaError(FA_ERR_UNSUPPORTED, f"dtype {t.dtype} (float16, bfloat16 or float32)")


def _need_cuda_contig(**ts):
    for name, t in ts.items():
        if t is None:
            continue
        if not t.is_cuda:
            raise FaError(FA_ERR_INVALID_ARG, f"{name} must be a CUDA tensor")
        if not t.is_contiguous():
            raise FaError(FA_ERR_INVALID_ARG, f"{name} must be contiguous")


def fa_last_error_string():
    return lib().fa_last_error_string().decode()


def fa_version():
    return lib().fa_version()


def fa_fwd_block_m():
    return lib().fa_fwd_block_m()


def fa_fwd_default_block_m(mask_mode):
    return lib().fa_fwd_default_block_m(mask_mode)


def fa_fwd_workspace_size(B, H, Sq, Sk, d, dtype):
    return lib().fa_fwd_workspace_size(B, H, Sq, Sk, d, dtype)


def fa_bwd_workspace_size(B, H, Sq):
    return lib().fa_bwd_workspace_size(B, H, Sq)


def fa_bwd(q, k, v, o, dout, lse, dq, dk, dv, workspace, scale, mask_mode=FA_MASK_NONE,
           window=0, n_global=0, stream=None, block_layout=None):
    """Gradients dq, dk, dv of fa_fwd for the upstream gradient dout (all [B,H,S,d]
    CUDA tensors of one 16-bit dtype; lse the float32 [B,H,Sq] fa_fwd returned; workspace
    a CUDA byte tensor of fa_bwd_workspace_size(B, H, Sq) bytes). FA_MASK_BLOCK_SPARSE takes
    block_layout, the uint8 CUDA layout of the forward call (fa_bwd_block_sparse)."""
    _need_cuda_contig(q=q, k=k, v=v, o=o, dout=dout, lse=lse, dq=dq, dk=dk, dv=dv,
                      workspace=workspace, block_layout=block_layout)
    B, H, Sq, d = q.shape
    if mask_mode == FA_MASK_BLOCK_SPARSE:
        _check(lib().fa_bwd_block_sparse(
            q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), dout.data_ptr(),
            lse.data_ptr(), dq.data_ptr(), dk.data_ptr(), dv.data_ptr(), workspace.data_ptr(),
            workspace.numel() * workspace.element_size(), B, H, Sq, k.shape[2], d, float(scale),
            _ptr(block_layout), _dtype_code(q), _stream(stream)))
        return
    _check(lib().fa_bwd(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), dout.data_ptr(),
                        lse.data_ptr(), dq.data_ptr(), dk.data_ptr(), dv.data_ptr(),
                        workspace.data_ptr(), workspace.numel() * workspace.element_size(), B,
                        H, Sq, k.shape[2], d, float(scale), mask_mode, window, n_global,
                        _dtype_code(q), _stream(stream)))


def fa_bwd_block_sparse(q, k, v, o, dout, lse, dq, dk, dv, workspace, scale, block_layout,
                        stream=None):
    """fa_bwd under FA_MASK_BLOCK_SPARSE with the forward call's device layout."""
    fa_bwd(q, k, v, o, dout, lse, dq, dk, dv, workspace, scale, FA_MASK_BLOCK_SPARSE,
           stream=stream, block_layout=block_layout)


def fa_fwd(q, k, v, o, lse, scale, mask_mode=FA_MASK_NONE, window=0, n_global=0, stream=None):
    """O = softmax(scale Q K^T + mask) V into `o` (and LSE into `lse`, may be None).

    q [B,H,Sq,d], k/v [B,H,Sk,d], o like q, lse float32 [B,H,Sq]; CUDA, contiguous.
    float32 inputs go through fa_fwd_ex, which needs a workspace (allocated here).
    """
    if q.dtype == torch.float32:
        return fa_fwd_ex(q, k, v, o, lse, scale, mask_mode, window, n_global, stream=stream)
    _need_cuda_contig(q=q, k=k, v=v, o=o, lse=lse)
    B, H, Sq, d = q.shape
    Sk = k.shape[2]
    _check(lib().fa_fwd(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), _ptr(lse), B, H,
                        Sq, Sk, d, float(scale), mask_mode, window, n_global, _dtype_code(q),
                        _stream(stream)))


def fa_fwd_ex(q, k, v, o, lse, scale, mask_mode=FA_MASK_NONE, window=0, n_global=0,
              block_n=0, block_m=0, num_ctas=0, group_heads=0, timeout_us=0, trace=None,
              block_layout=None, workspace=None, rescale_count=None, stream=None,
              block_layout_host=None):
    """fa_fwd with the tuning and debug fields of fa_fwd_params. block_layout: uint8 CUDA
    tensor [H, ceil(Sq/128), ceil(Sk/128)] for FA_MASK_BLOCK_SPARSE; block_layout_host:
    the same layout as a contiguous CPU uint8 tensor, for the work plan. workspace: CUDA byte
    tensor of fa_fwd_workspace_size(...) bytes for float32 inputs (allocated here when
    None). rescale_count: zeroed int32 CUDA tensor [B*H, ceil(Sq/128)] that counts the
    rows whose output was rescaled, per 128-query tile."""
    _need_cuda_contig(q=q, k=k, v=v, o=o, lse=lse, trace=trace, block_layout=block_layout,
                      workspace=workspace, rescale_count=rescale_count)
    B, H, Sq, d = q.shape
    dt = _dtype_code(q)
    if workspace is None and dt == FA_F32:
        workspace = torch.empty(max(fa_fwd_workspace_size(B, H, Sq, k.shape[2], d, dt), 16),
                                dtype=torch.uint8, device=q.device)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    if block_layout_host is not None:
        want = (H, -(-Sq // 128), -(-k.shape[2] // 128))
        if (block_layout_host.device.type != "cpu" or block_layout_host.dtype != torch.uint8
                or not block_layout_host.is_contiguous()
                or tuple(block_layout_host.shape) != want):
            raise ValueError(f"block_layout_host must be a contiguous CPU uint8 tensor {want}")
    p = FwdParams(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), _ptr(lse), B, H, Sq,
                  k.shape[2], d, float(scale), mask_mode, window, n_global, dt,
                  block_n, block_m, num_ctas, group_heads, timeout_us, _ptr(trace),
                  _ptr(block_layout), _ptr(workspace), ws_bytes, _ptr(rescale_count),
                  None if block_layout_host is None else block_layout_host.data_ptr())
    _check(lib().fa_fwd_ex(ctypes.byref(p), _stream(stream)))


def fa_decode_workspace_size(B, H, d, max_pages_per_seq, page_size):
    return lib().fa_decode_workspace_size(B, H, d, max_pages_per_seq, page_size)


def fa_decode_default_pages_per_split(B, H, max_pages_per_seq):
    return lib().fa_decode_default_pages_per_split(B, H, max_pages_per_seq)


def fa_decode_paged(q, k_pages, v_pages, block_table, ctx_lens, o, lse, scale, workspace,
                    stream=None):
    """One query token per sequence against a paged KV cache.

    q/o [B,H,d]; pools [num_pages,H,page_size,d]; block_table int32 [B,max_pages];
    ctx_lens int32 [B]; lse float32 [B,H] or None; workspace a CUDA byte tensor.
    """
    _need_cuda_contig(q=q, k_pages=k_pages, v_pages=v_pages, block_table=block_table,
                      ctx_lens=ctx_lens, o=o, lse=lse, workspace=workspace)
    B, H, d = q.shape
    P, _, page, _ = k_pages.shape
    _check(lib().fa_decode_paged(q.data_ptr(), k_pages.data_ptr(), v_pages.data_ptr(),
                                 block_table.data_ptr(), ctx_lens.data_ptr(), o.data_ptr(),
                                 _ptr(lse), B, H, d, page, block_table.shape[1], P, float(scale),
                                 _dtype_code(q), workspace.data_ptr(),
                                 workspace.numel() * workspace.element_size(), _stream(stream)))


def fa_decode_paged_ex(q, k_pages, v_pages, block_table, ctx_lens, o, lse, scale, workspace,
                       pages_per_split=0, trace_pages=None, trace_splits=None, stream=None):
    _need_cuda_contig(q=q, k_pages=k_pages, v_pages=v_pages, block_table=block_table,
                      ctx_lens=ctx_lens, o=o, lse=lse, workspace=workspace,
                      trace_pages=trace_pages, trace_splits=trace_splits)
    B, H, d = q.shape
    P, _, page, _ = k_pages.shape
    p = DecodeParams(q.data_ptr(), k_pages.data_ptr(), v_pages.data_ptr(), block_table.data_ptr(),
                     ctx_lens.data_ptr(), o.data_ptr(), _ptr(lse), B, H, d, page,
                     block_table.shape[1], P, float(scale), _dtype_code(q), workspace.data_ptr(),
                     workspace.numel() * workspace.element_size(), pages_per_split,
                     _ptr(trace_pages), _ptr(trace_splits))
    _check(lib().fa_decode_paged_ex(ctypes.byref(p), _stream(stream)))


def fa_decode_paged_noalloc(q, k_pages, v_pages, block_table, ctx_lens, o, lse, scale,
                            stream=None):
    """fa_decode_paged for callers that cannot allocate a workspace: the split partials
    go to a fixed 16 MiB scratch array inside the library (one per GPU). Calls that
    overlap on the GPU share that array and race; the first call on a device should
    come before any stream capture."""
    _need_cuda_contig(q=q, k_pages=k_pages, v_pages=v_pages, block_table=block_table,
                      ctx_lens=ctx_lens, o=o, lse=lse)
    B, H, d = q.shape
    P, _, page, _ = k_pages.shape
    _check(lib().fa_decode_paged_noalloc(q.data_ptr(), k_pages.data_ptr(), v_pages.data_ptr(),
                                         block_table.data_ptr(), ctx_lens.data_ptr(),
                                         o.data_ptr(), _ptr(lse), B, H, d, page,
                                         block_table.shape[1], P, float(scale), _dtype_code(q),
                                         _stream(stream)))


def fa_fwd_paged(q, k_pages, v_pages, block_table, ctx_lens, o, lse, scale,
                 mask_mode=FA_MASK_CAUSAL, window=0, n_global=0, stream=None,
                 ctx_lens_host=None):
    """Chunked prefill against a paged cache: q/o [B,H,Sq,d] are the last Sq tokens of
    each sequence; pools [num_pages,H,page,d]; block_table int32 [B,max_pages];
    ctx_lens int32 [B] (cached tokens, the chunk included). ctx_lens_host: the same
    lengths as a CPU int32 tensor, for the work plan (fa_fwd_paged_host_lens)."""
    _need_cuda_contig(q=q, k_pages=k_pages, v_pages=v_pages, block_table=block_table,
                      ctx_lens=ctx_lens, o=o, lse=lse)
    B, H, Sq, d = q.shape
    P, _, page, _ = k_pages.shape
    if ctx_lens_host is None:
        _check(lib().fa_fwd_paged(q.data_ptr(), k_pages.data_ptr(), v_pages.data_ptr(),
                                  block_table.data_ptr(), ctx_lens.data_ptr(), o.data_ptr(),
                                  _ptr(lse), B, H, Sq, d, page, block_table.shape[1], P,
                                  float(scale), mask_mode, window, n_global, _dtype_code(q),
                                  _stream(stream)))
        return
    if (ctx_lens_host.device.type != "cpu" or ctx_lens_host.dtype != torch.int32
            or not ctx_lens_host.is_contiguous() or ctx_lens_host.numel() != B):
        raise ValueError("ctx_lens_host must be a contiguous CPU int32 tensor of B entries")
    _check(lib().fa_fwd_paged_host_lens(q.data_ptr(), k_pages.data_ptr(), v_pages.data_ptr(),
                                        block_table.data_ptr(), ctx_lens.data_ptr(),
                                        ctx_lens_host.data_ptr(), o.data_ptr(), _ptr(lse), B, H,
                                        Sq, d, page, block_table.shape[1], P, float(scale),
                                        mask_mode, window, n_global, _dtype_code(q),
                                        _stream(stream)))


def fa_fwd_paged_host_lens(q, k_pages, v_pages, block_table, ctx_lens, ctx_lens_host, o, lse,
                           scale, mask_mode=FA_MASK_CAUSAL, window=0, n_global=0, stream=None):
    """fa_fwd_paged with the lengths also in host memory (a CPU int32 tensor) for the plan."""
    fa_fwd_paged(q, k_pages, v_pages, block_table, ctx_lens, o, lse, scale, mask_mode, window,
                 n_global, stream, ctx_lens_host=ctx_lens_host)


def fa_kv_append(k_new, v_new, k_pages, v_pages, block_table, ctx_lens, new_lens=None,
                 stream=None):
    """Write k_new/v_new [B,H,T,d] at positions ctx_lens[b] + t of the paged cache
    (t < new_lens[b], or all T); zero-fill the rest of each chunk's last page."""
    _need_cuda_contig(k_new=k_new, v_new=v_new, k_pages=k_pages, v_pages=v_pages,
                      block_table=block_table, ctx_lens=ctx_lens, new_lens=new_lens)
    B, H, T, d = k_new.shape
    P, _, page, _ = k_pages.shape
    _check(lib().fa_kv_append(k_new.data_ptr(), v_new.data_ptr(), k_pages.data_ptr(),
                              v_pages.data_ptr(), block_table.data_ptr(), ctx_lens.data_ptr(),
                              _ptr(new_lens), B, H, T, d, page, block_table.shape[1], P,
                              _dtype_code(k_new), _stream(stream)))


def fa_merge_partials(o_a, lse_a, o_b, lse_b, o, lse=None, stream=None):
    """Combine two attention results over disjoint key sets of the same queries by LSE.

    o_* [..., d] (same shape, fp16/bf16), lse_* float32 with the leading shape of o.
    """
    _need_cuda_contig(o_a=o_a, lse_a=lse_a, o_b=o_b, lse_b=lse_b, o=o, lse=lse)
    d = o_a.shape[-1]
    rows = o_a.numel() // d
    _check(lib().fa_merge_partials(o_a.data_ptr(), lse_a.data_ptr(), o_b.data_ptr(),
                                   lse_b.data_ptr(), o.data_ptr(), _ptr(lse), rows, d,
                                   _dtype_code(o_a), _stream(stream)))


def fa_get_device_status(stream=None):
    """Synchronise the stream, read and clear the device status word; returns the code."""
    return lib().fa_get_device_status(_stream(stream))


def fa_selftest_timeout(timeout_us, stream=None):
    _check(lib().fa_selftest_timeout(timeout_us, _stream(stream)))


# ----------------------------------------------------------- packed tokens, grouped heads

def _refuse(msg):
    raise FaError(FA_ERR_INVALID_ARG, msg)


def _int32(**values):
    """Refuse what a C int does not hold: ctypes would cut it to its low 32 bits."""
    for name, x in values.items():
        try:
            ok = -2 ** 31 <= operator.index(x) < 2 ** 31
        except TypeError:
            ok = False
        if not ok:
            _refuse(f"{name} = {x!r} is not a 32-bit integer")


def _packer(cls):
    """The bytes of a parameter struct from its values in order: a Structure's constructor costs
    several times as much (1.2 us against 0.2)."""
    code = {_vp: "P", _i64: "q", _i: "i", _f: "f", _sz: "N", _u32: "I"}
    pack = struct.Struct("@" + "".join(code[t] for _, t in cls._fields_)).pack

    def checked(*values):
        try:
            return pack(*values)
        except (struct.error, OverflowError):  # which value was it?
            for (name, t), x in zip(cls._fields_, values):
                try:
                    struct.pack(code[t], x)
                except (struct.error, OverflowError) as e:
                    _refuse(f"{name} = {x!r}: {e}")
            raise
    return checked


_pack_append = _packer(RopeAppendParams)
_pack_varlen = _packer(VarlenParams)
_pack_grads = _packer(VarlenGrads)
_pack_paged = _packer(PagedVarlenParams)


def _rows(name, t, n, heads, d, dtype, device):
    """Elements between the tokens of packed rows [n, heads, d] (a view of a wider row is fine:
    the last two dimensions have to be dense)."""
    if t.dtype is dtype and t.device == device and n > 1 and t.shape == (n, heads, d):
        st = t.stride()
        if st[2] == 1 and st[1] == d:
            return st[0]
    return _rows_checked(name, t, n, heads, d, dtype, device)


def _rows_checked(name, t, n, heads, d, dtype, device):
    if t.shape != (n, heads, d) or t.dtype != dtype or t.device != device:
        _refuse(f"{name} must be [{n}, {heads}, {d}] of {dtype} on {device}, not "
                f"{list(t.shape)} of {t.dtype} on {t.device}")
    st = t.stride()
    if n == 0:
        return heads * d
    if (d > 1 and st[2] != 1) or (heads > 1 and st[1] != d):
        _refuse(f"{name}: the heads of a token must lie next to each other")
    return st[0] if n > 1 else heads * d


def _dims(name, t, n):
    """The shape of t, which must have n dimensions."""
    shape = t.shape
    if len(shape) != n:
        _refuse(f"{name} must have {n} dimensions, not {len(shape)}")
    return shape


def _ints(name, t, shape, device):
    if t.dtype is not torch.int32 or t.shape != shape or t.device != device \
            or not t.is_contiguous():
        _refuse(f"{name} must be a contiguous int32 tensor {shape} on {device}")
    return t.data_ptr()


def _packed_device(t):
    """The device of t, which must be the current one: the library launches there."""
    if not t.is_cuda:
        _refuse("tensors must be CUDA tensors")
    if t.device.index != torch.cuda.current_device():
        _refuse(f"tensors are on {t.device}, the current device is "
                f"cuda:{torch.cuda.current_device()}")
    return t.device


def _lse_ptr(lse, n, heads, device):
    if lse is None:
        return 0
    if lse.dtype != torch.float32 or lse.device != device or not lse.is_contiguous() \
            or tuple(lse.shape) != (n, heads):
        _refuse(f"lse must be a contiguous float32 tensor ({n}, {heads}) on {device}")
    return lse.data_ptr()


def _bytes_of(workspace, device):
    if workspace.device != device or not workspace.is_contiguous():
        _refuse(f"workspace must be a contiguous tensor on {device}")
    return workspace.data_ptr(), workspace.numel() * workspace.element_size()


def fa_rope_freqs(rot_dim, base=10000.0, scaling=FA_ROPE_PLAIN, factor=1.0, trained_len=0,
                  fast=32.0, slow=1.0, device=None):
    """(frequencies float64 [rot_dim/2] in radians per position, amplitude) of a rotary
    embedding; the rules are those of fa_rope_freqs in fa.h. On `device` (CPU when None)."""
    _int32(rot_dim=rot_dim, scaling=scaling, trained_len=trained_len)
    host = torch.empty(min(max(rot_dim // 2, 1), 256), dtype=torch.float64)  # 512 is the largest
    amp = _f()
    _check(lib().fa_rope_freqs(ctypes.cast(host.data_ptr(), ctypes.POINTER(ctypes.c_double)),
                               ctypes.byref(amp), rot_dim, float(base), scaling, float(factor),
                               trained_len, float(fast), float(slow)))
    return (host if device is None else host.to(device)), amp.value


def _freqs_ptr(freqs, device):
    if freqs.dtype != torch.float64 or freqs.device != device or freqs.dim() != 1 \
            or not freqs.is_contiguous():
        _refuse(f"freqs must be a contiguous float64 vector on {device}")
    return freqs.data_ptr()


def fa_rope(x, y, positions, freqs, style=FA_ROPE_HALF, amplitude=1.0, inverse=False,
            stream=None):
    """y = x [T, H, d] with the first 2 * len(freqs) elements of every head rotated by
    positions (int32 [T]) * freqs; y may be x. inverse=True turns back: the gradient of x
    from the gradient of y. float16, bfloat16 or float32; any token and head steps."""
    device = _packed_device(x)
    if x.dim() != 3 or y.shape != x.shape or y.dtype != x.dtype or y.device != device:
        _refuse("x and y must be [tokens, heads, d] of one dtype on one device")
    T, H, d = x.shape
    if T == 0 or H == 0:
        return
    xs, ys = x.stride(), y.stride()
    if d > 1 and (xs[2] != 1 or ys[2] != 1):
        _refuse("the elements of a head must be contiguous")
    dense, rot = H * d, 2 * freqs.numel()
    if H >= 2 ** 31 or d >= 2 ** 31 or rot >= 2 ** 31:
        _int32(heads=H, head_dim=d, rot_dim=rot)
    if style != FA_ROPE_HALF and style != FA_ROPE_PAIRS:
        _refuse(f"style {style}")
    _check(lib().fa_rope(x.data_ptr(), y.data_ptr(), _ints("positions", positions, (T,), device),
                         _freqs_ptr(freqs, device), T, H, d, rot,
                         xs[0] if T > 1 else dense, xs[1] if H > 1 else d,
                         ys[0] if T > 1 else dense, ys[1] if H > 1 else d,
                         style, float(amplitude), 1 if inverse else 0, _dtype_code(x),
                         _stream(stream)))


def fa_rope_append(q, k, v, q_out, k_pages, v_pages, block_table, ctx_lens, cu_seqlens, freqs,
                   style=FA_ROPE_HALF, amplitude=1.0, stream=None):
    """Rotate q and k of a packed chunk (q, q_out [T, H, d]; k, v [T, Hkv, d]) by the tokens'
    positions ctx_lens[b] + t - cu_seqlens[b] (ctx_lens: tokens cached before the chunk), write
    q to q_out and k and v into the pools [num_pages, Hkv, page_size, d]."""
    device = _packed_device(q)
    T, H, d = _dims("q", q, 3)
    P, Hkv, page, _ = _dims("k_pages", k_pages, 4)
    B, width = _dims("block_table", block_table, 2)
    _pools(k_pages, v_pages, d, q.dtype, device)
    p = _pack_append(
        q.data_ptr(), k.data_ptr(), v.data_ptr(), q_out.data_ptr(), k_pages.data_ptr(),
        v_pages.data_ptr(), _ints("block_table", block_table, (B, width), device),
        _ints("ctx_lens", ctx_lens, (B,), device),
        _ints("cu_seqlens", cu_seqlens, (B + 1,), device), _freqs_ptr(freqs, device),
        _rows("q", q, T, H, d, q.dtype, device), _rows("k", k, T, Hkv, d, q.dtype, device),
        _rows("v", v, T, Hkv, d, q.dtype, device),
        _rows("q_out", q_out, T, H, d, q.dtype, device),
        T, B, H, Hkv, d, 2 * freqs.numel(), page, width, P, style, float(amplitude),
        _dtype_code(q))
    _check(lib().fa_rope_append(p, _stream(stream)))


def _pools(k_pages, v_pages, d, dtype, device):
    for name, t in (("k_pages", k_pages), ("v_pages", v_pages)):
        if t.dtype != dtype or t.device != device or not t.is_contiguous() \
                or t.shape != k_pages.shape or t.shape[3] != d:
            _refuse(f"{name} must be contiguous [num_pages, Hkv, page_size, {d}] of {dtype} on "
                    f"{device}")


def fa_varlen_workspace_size(B, H, Hkv, total_q, total_k, d):
    _int32(B=B, H=H, Hkv=Hkv, total_q=total_q, total_k=total_k, d=d)
    return lib().fa_varlen_workspace_size(B, H, Hkv, total_q, total_k, d)


def fa_bwd_varlen_workspace_size(B, H, Hkv, total_q, total_k, d):
    _int32(B=B, H=H, Hkv=Hkv, total_q=total_q, total_k=total_k, d=d)
    return lib().fa_bwd_varlen_workspace_size(B, H, Hkv, total_q, total_k, d)


def fa_paged_varlen_workspace_size(B, H, Hkv, total_q, max_q, max_pages_per_seq, page_size, d):
    _int32(B=B, H=H, Hkv=Hkv, total_q=total_q, max_q=max_q, max_pages_per_seq=max_pages_per_seq,
           page_size=page_size, d=d)
    return lib().fa_paged_varlen_workspace_size(B, H, Hkv, total_q, max_q, max_pages_per_seq,
                                                page_size, d)


def _varlen(q, k, v, o, lse, cu_seqlens_q, cu_seqlens_k, scale, workspace, mask_mode, window,
            n_global):
    device = _packed_device(q)
    Tq, H, d = _dims("q", q, 3)
    Tk, Hkv, _ = _dims("k", k, 3)
    B = cu_seqlens_q.numel() - 1
    ws, ws_bytes = _bytes_of(workspace, device)
    return _pack_varlen(
        q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), _lse_ptr(lse, Tq, H, device),
        _rows("q", q, Tq, H, d, q.dtype, device), _rows("k", k, Tk, Hkv, d, q.dtype, device),
        _rows("v", v, Tk, Hkv, d, q.dtype, device), _rows("o", o, Tq, H, d, q.dtype, device),
        _ints("cu_seqlens_q", cu_seqlens_q, (B + 1,), device),
        _ints("cu_seqlens_k", cu_seqlens_k, (B + 1,), device), B, H, Hkv, d, Tq, Tk,
        float(scale), mask_mode, window, n_global, _dtype_code(q), ws, ws_bytes, 0)


def fa_fwd_varlen(q, k, v, o, lse, cu_seqlens_q, cu_seqlens_k, scale, workspace,
                  mask_mode=FA_MASK_CAUSAL, window=0, n_global=0, stream=None):
    """Attention over packed sequences: q, o [Tq, H, d], k, v [Tk, Hkv, d] (slices of wider rows
    are fine), cu_seqlens_* int32 [B + 1], lse float32 [Tq, H] or None; query head h reads K/V
    head h // (H // Hkv). workspace: a CUDA byte tensor of fa_varlen_workspace_size(...)."""
    p = _varlen(q, k, v, o, lse, cu_seqlens_q, cu_seqlens_k, scale, workspace, mask_mode, window,
                n_global)
    _check(lib().fa_fwd_varlen(p, _stream(stream)))


def fa_bwd_varlen(q, k, v, o, dout, lse, dq, dk, dv, cu_seqlens_q, cu_seqlens_k, scale,
                  workspace, mask_mode=FA_MASK_CAUSAL, window=0, n_global=0, stream=None):
    """Gradients dq [Tq, H, d], dk, dv [Tk, Hkv, d] of fa_fwd_varlen for the upstream gradient
    dout; o and lse as the forward call wrote them. workspace: a CUDA byte tensor of
    fa_bwd_varlen_workspace_size(...)."""
    if lse is None:
        _refuse("the backward needs the forward's lse")
    p = _varlen(q, k, v, o, lse, cu_seqlens_q, cu_seqlens_k, scale, workspace, mask_mode, window,
                n_global)
    Tq, H, d = q.shape
    Tk, Hkv, _ = k.shape
    g = _pack_grads(dout.data_ptr(), dq.data_ptr(), dk.data_ptr(), dv.data_ptr(),
                    _rows("dout", dout, Tq, H, d, q.dtype, q.device),
                    _rows("dq", dq, Tq, H, d, q.dtype, q.device),
                    _rows("dk", dk, Tk, Hkv, d, q.dtype, q.device),
                    _rows("dv", dv, Tk, Hkv, d, q.dtype, q.device))
    _check(lib().fa_bwd_varlen(p, g, _stream(stream)))


def fa_fwd_paged_varlen(q, k_pages, v_pages, block_table, ctx_lens, cu_seqlens_q, max_q, o, lse,
                        scale, workspace, mask_mode=FA_MASK_CAUSAL, window=0, n_global=0,
                        stream=None):
    """Attention of packed chunks of new tokens (the last tokens of their sequences) over a
    paged cache: q, o [Tq, H, d]; pools [num_pages, Hkv, page_size, d]; block_table int32
    [B, max_pages]; ctx_lens int32 [B] (cached keys, the chunk's included); max_q at least the
    longest chunk. workspace: a CUDA byte tensor of fa_paged_varlen_workspace_size(...)."""
    device = _packed_device(q)
    Tq, H, d = _dims("q", q, 3)
    P, Hkv, page, _ = _dims("k_pages", k_pages, 4)
    B, width = _dims("block_table", block_table, 2)
    _pools(k_pages, v_pages, d, q.dtype, device)
    ws, ws_bytes = _bytes_of(workspace, device)
    p = _pack_paged(
        q.data_ptr(), k_pages.data_ptr(), v_pages.data_ptr(),
        _ints("block_table", block_table, (B, width), device),
        _ints("ctx_lens", ctx_lens, (B,), device),
        _ints("cu_seqlens_q", cu_seqlens_q, (B + 1,), device), o.data_ptr(),
        _lse_ptr(lse, Tq, H, device), _rows("q", q, Tq, H, d, q.dtype, device),
        _rows("o", o, Tq, H, d, q.dtype, device), B, H, Hkv, d, Tq, max_q, page, width, P,
        float(scale), mask_mode, window, n_global, _dtype_code(q), ws, ws_bytes, 0)
    _check(lib().fa_fwd_paged_varlen(p, _stream(stream)))
