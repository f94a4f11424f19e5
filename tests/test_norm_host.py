"""Refusals of the calls with norms, several axes, an 8-bit cache and trees, and the host-side axis
map: no GPU. Fake addresses throughout; a refused call launches nothing."""
import ctypes
import math

import pytest
import torch

import _cache8 as c8
import tiled_attention_06_gb300 as fa
from tiled_attention_06_gb300 import build as fa_build

A = 1 << 20  # a 16-byte-aligned fake address
OK, INVALID, UNSUPPORTED = fa.FA_OK, fa.FA_ERR_INVALID_ARG, fa.FA_ERR_UNSUPPORTED


@pytest.fixture(scope="module")
def L():
    fa_build.build()
    return fa.lib()


def fill(cls, base, kw):
    a = dict(base, **kw)
    return cls(*[a[f] for f, _ in cls._fields_])


# ------------------------------------------------------------------ which axis turns which pair

@pytest.mark.parametrize("sections,turns,want", [
    ([4], False, [0] * 4), ([2, 1, 3], False, [0, 0, 1, 2, 2, 2]),
    ([2, 1, 3], True, [0, 1, 2, 0, 2, 2]), ([0, 2, 0, 1], True, [1, 3, 1]),
    ([2, 2], True, [0, 1, 0, 1]), ([1, 0], False, [0])], ids=str)
def test_axes(L, sections, turns, want):
    assert fa.fa_rope_axes(sections, turns).tolist() == want


@pytest.mark.parametrize("sections", [[], [0], [0, 0], [-1, 3], [1] * 5, [257], [2 ** 40]], ids=str)
def test_axes_refusals(L, sections):
    with pytest.raises(fa.FaError) as e:
        fa.fa_rope_axes(sections)
    assert e.value.status == INVALID


def test_axes_refuses_a_wrong_sum(L):
    out, three = torch.zeros(8, dtype=torch.int32), torch.tensor([3], dtype=torch.int32)
    assert L.fa_rope_axes(out.data_ptr(), 8, three.data_ptr(), 1, 0) == INVALID
    assert L.fa_rope_axes(None, 6, three.data_ptr(), 1, 0) == INVALID
    assert L.fa_rope_axes(out.data_ptr(), 7, three.data_ptr(), 1, 0) == INVALID


# ------------------------------------------------------------------ fa_norm_rope and its gradient

NORM = dict(q=A, k=A, q_out=2 * A, k_out=2 * A, positions=A, pair_axis=A, freqs=A, q_weight=A,
            k_weight=A, T=4, q_token=128, q_head=64, k_token=64, k_head=64, q_out_token=128,
            q_out_head=64, k_out_token=64, k_out_head=64, H=2, Hkv=1, d=64, rot_dim=64, axes=3,
            style=0, amplitude=1.0, norm=1, eps=1e-6, weight_dtype=0, dtype=0)
TURNS = [
    (dict(d=1), INVALID), (dict(d=514, q_head=514), INVALID), (dict(d=63), UNSUPPORTED),
    (dict(rot_dim=0), INVALID), (dict(rot_dim=66), INVALID), (dict(rot_dim=5), INVALID),
    (dict(axes=0), INVALID), (dict(axes=5), INVALID), (dict(style=2), INVALID),
    (dict(amplitude=math.inf), INVALID), (dict(norm=2), INVALID), (dict(eps=-1e-9), INVALID),
    (dict(eps=math.nan), INVALID), (dict(weight_dtype=1), INVALID), (dict(dtype=3), UNSUPPORTED),
    (dict(q_weight=A + 1), INVALID), (dict(weight_dtype=2, k_weight=A + 2), INVALID),
    (dict(freqs=None), INVALID), (dict(freqs=A + 4), INVALID), (dict(positions=A + 2), INVALID),
    (dict(pair_axis=None), INVALID), (dict(pair_axis=A + 2), INVALID)]


@pytest.mark.parametrize("kw,want", TURNS + [
    (dict(T=0, q=None), OK), (dict(T=-1), INVALID), (dict(H=0), INVALID), (dict(Hkv=-1), INVALID),
    (dict(positions=None), INVALID), (dict(q=None), INVALID), (dict(k_out=None), INVALID),
    (dict(q=A + 1), INVALID), (dict(dtype=2, weight_dtype=2, k=A + 2), INVALID),
    (dict(q_head=60), INVALID), (dict(q_out_token=64), INVALID), (dict(k_token=-64), INVALID),
    (dict(q_out=A, q_out_token=256), INVALID), (dict(k_out=A, k_out_head=128), INVALID),
    (dict(T=1 << 34), INVALID)], ids=str)
def test_norm_rope_refusals(L, kw, want):
    assert L.fa_norm_rope(ctypes.byref(fill(fa.NormRopeParams, NORM, kw)), None) == want


GRADS = dict(dq_out=A, dk_out=A, dq=2 * A, dk=2 * A, dq_weight=A, dk_weight=A, dq_out_token=128,
             dq_out_head=64, dk_out_token=64, dk_out_head=64, dq_token=128, dq_head=64, dk_token=64,
             dk_head=64, workspace=A, workspace_bytes=1 << 40)


@pytest.mark.parametrize("kw,g,want", [(k, {}, w) for k, w in TURNS] + [
    (dict(q=None), {}, INVALID), (dict(k=A + 1), {}, INVALID), (dict(positions=None), {}, INVALID),
    ({}, dict(dq_out=None), INVALID), ({}, dict(dk=A + 1), INVALID), ({}, dict(dq_token=64), INVALID),
    ({}, dict(dq=A, dq_token=256), INVALID), ({}, dict(dq_weight=A + 2), INVALID),
    ({}, dict(workspace=None), INVALID), ({}, dict(workspace=A + 8), INVALID),
    ({}, dict(workspace_bytes=64), INVALID),
    (dict(norm=0), {}, INVALID)], ids=str)  # a weight's gradient without a norm
def test_norm_rope_gradient_refusals(L, kw, g, want):
    assert L.fa_norm_rope_bwd(ctypes.byref(fill(fa.NormRopeParams, NORM, kw)),
                              ctypes.byref(fill(fa.NormRopeGrads, GRADS, g)), None) == want


def test_null_structs(L):
    n = ctypes.byref(fill(fa.NormRopeParams, NORM, {}))
    p = ctypes.byref(fill(fa.PagedVarlenParams, PAGED, {}))
    assert L.fa_norm_rope(None, None) == L.fa_norm_rope_bwd(n, None, None) == INVALID
    assert L.fa_norm_rope_append(None, None) == L.fa_kv_read(None, None) == INVALID
    assert L.fa_fwd_paged_varlen_ex(p, None, None) == INVALID
    assert L.fa_norm_rope_bwd_workspace_size(0, 1, 64) == 0
    assert L.fa_norm_rope_bwd_workspace_size(1, 0, 1024) == 0


# ------------------------------------------------------------------ the cache

APPEND = dict(q=A, k=A, v=A, q_out=A, k_pages=A, v_pages=A, k_scales=A, v_scales=A, block_table=A,
              ctx_lens=A, cu_seqlens=A, positions=A, pair_axis=A, freqs=A, q_weight=A, k_weight=A,
              q_token=256, k_token=128, v_token=128, q_out_token=256, T=5, B=2, H=4, Hkv=2, d=64,
              rot_dim=64, axes=2, page_size=16, max_pages_per_seq=4, num_pages=8, style=0,
              amplitude=1.0, norm=1, eps=1e-6, weight_dtype=0, dtype=0)


@pytest.mark.parametrize("kw,want", [t for t in TURNS if "q_head" not in t[0]] + [
    (dict(T=0, q=None), OK), (dict(T=-1), INVALID), (dict(B=0), INVALID), (dict(d=96), UNSUPPORTED),
    (dict(dtype=2, weight_dtype=2), UNSUPPORTED), (dict(page_size=24), UNSUPPORTED),
    (dict(q=None), INVALID), (dict(k=A + 8), INVALID), (dict(v_token=120), INVALID),
    (dict(k_token=132), INVALID), (dict(q_out_token=264), INVALID), (dict(k_pages=None), INVALID),
    (dict(v_pages=A + 8), INVALID), (dict(block_table=None), INVALID), (dict(ctx_lens=A + 2), INVALID),
    (dict(k_scales=None), INVALID), (dict(v_scales=None), INVALID), (dict(positions=None), INVALID),
    (dict(num_pages=0), INVALID), (dict(page_size=4096, max_pages_per_seq=1 << 20), INVALID)], ids=str)
def test_append_refusals(L, kw, want):
    assert L.fa_norm_rope_append(ctypes.byref(fill(fa.NormRopeAppendParams, APPEND, kw)), None) == want


READ = dict(k_pages=A, v_pages=A, k_scales=A, v_scales=A, block_table=A, starts=A, cu_seqlens=A, k=A,
            v=A, k_token=128, v_token=128, T=5, B=2, Hkv=2, d=64, page_size=16, max_pages_per_seq=4,
            num_pages=8, dtype=0)


@pytest.mark.parametrize("kw,want", [
    (dict(T=0, k=None), OK), (dict(T=-1), INVALID), (dict(dtype=2), UNSUPPORTED),
    (dict(d=96), UNSUPPORTED), (dict(page_size=8), UNSUPPORTED), (dict(B=0), INVALID),
    (dict(k=None), INVALID), (dict(v=A + 8), INVALID), (dict(k_token=64), INVALID),
    (dict(k_pages=None), INVALID), (dict(k_scales=None), INVALID), (dict(v_scales=None), INVALID),
    (dict(starts=None), INVALID), (dict(starts=A + 2), INVALID), (dict(cu_seqlens=None), INVALID),
    (dict(block_table=A + 1), INVALID)], ids=str)
def test_read_refusals(L, kw, want):
    assert L.fa_kv_read(ctypes.byref(fill(fa.KvReadParams, READ, kw)), None) == want


PAGED = dict(q=A, k_pages=A, v_pages=A, block_table=A, ctx_lens=A, cu_seqlens_q=A, o=A, lse=A,
             q_token=256, o_token=256, B=2, H=4, Hkv=2, d=64, total_q=10, max_q=8, page_size=16,
             max_pages_per_seq=4, num_pages=8, scale=0.125, mask_mode=1, window=0, n_global=0,
             dtype=0, workspace=A, workspace_bytes=1 << 40, timeout_us=0)
EXTRA = dict(k_scales=A, v_scales=A, tree=None, tree_words=0)


@pytest.mark.parametrize("kw,x,want", [
    (dict(total_q=0, q=None), {}, OK), (dict(total_q=0), dict(tree=A, tree_words=1), INVALID),
    ({}, dict(k_scales=None), INVALID), ({}, dict(v_scales=None), INVALID),
    ({}, dict(k_scales=A + 8), INVALID), (dict(mask_mode=6), {}, INVALID),
    (dict(mask_mode=7), {}, INVALID), (dict(mask_mode=5), {}, UNSUPPORTED),
    (dict(mask_mode=6), dict(tree=A, tree_words=0), INVALID),
    (dict(mask_mode=6), dict(tree=A + 2, tree_words=1), INVALID),
    (dict(mask_mode=6, max_q=33), dict(tree=A, tree_words=1), INVALID),
    (dict(mask_mode=6, total_q=0), dict(tree=A, tree_words=1), OK),
    (dict(d=96), {}, UNSUPPORTED), (dict(dtype=2), {}, UNSUPPORTED), (dict(scale=0.0), {}, INVALID),
    (dict(workspace_bytes=64), {}, INVALID), (dict(k_pages=A + 8), {}, INVALID),
    (dict(q_token=252), {}, INVALID)], ids=str)
def test_attention_refusals(L, kw, x, want):
    assert L.fa_fwd_paged_varlen_ex(ctypes.byref(fill(fa.PagedVarlenParams, PAGED, kw)),
                                    ctypes.byref(fill(fa.PagedVarlenExtra, EXTRA, x)), None) == want


def test_python_refuses_cpu_tensors():
    x = torch.zeros(3, 2, 64, dtype=torch.float16)
    with pytest.raises(fa.FaError):
        fa.fa_norm_rope(x, None, x, None, torch.zeros(1, 3, dtype=torch.int32), fa.fa_rope_freqs(64)[0])


# ------------------------------------------------------------------ the tests' own 8-bit form

def test_the_reference_rounds_as_the_type_does():
    """Every finite value and the middles between neighbours, against torch's conversion."""
    x = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).float()
    x = x[torch.isfinite(x)].sort().values
    x = torch.cat([x, (x[1:] + x[:-1]) / 2, torch.tensor([448.0])])
    x = torch.cat([x, torch.full((-len(x) % 2,), 448.0)]).view(-1, 1)
    x = torch.cat([x, torch.full_like(x, 448.0)], 1)  # every row needs the power 1
    got, power = c8.quantise(x)
    assert (power == 127).all()
    assert torch.equal(got, x.to(torch.float8_e4m3fn).view(torch.uint8))


@pytest.mark.parametrize("amax,byte", [(448.0, 127), (448.0001, 128), (224.0, 126), (1.0, 119),
                                       (0.0, 0), (1.75 * 2 ** -119, 0), (3e38, 247)])
def test_the_reference_takes_the_smallest_power(amax, byte):
    assert c8.exponent_byte(torch.tensor([amax], dtype=torch.float64)).item() == byte
