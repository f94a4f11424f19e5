"""Refusals of the calls over packed tokens, and the host-side frequencies: no GPU. Fake
addresses throughout; a refused call launches nothing."""
import ctypes
import math

import pytest
import torch

import tiled_attention_06_gb300 as fa
from tiled_attention_06_gb300 import build as fa_build

A = 1 << 20  # a 16-byte-aligned fake address
OK, INVALID, UNSUPPORTED = fa.FA_OK, fa.FA_ERR_INVALID_ARG, fa.FA_ERR_UNSUPPORTED


@pytest.fixture(scope="module")
def L():
    fa_build.build()
    return fa.lib()


# ------------------------------------------------------------------ frequencies

def test_frequency_rules():
    R, base = 64, 10000.0
    plain = [base ** (-2 * i / R) for i in range(R // 2)]
    w, a = fa.fa_rope_freqs(R)
    assert a == 1.0 and torch.allclose(w, torch.tensor(plain, dtype=torch.float64), rtol=1e-14)
    w, a = fa.fa_rope_freqs(R, scaling=fa.FA_ROPE_LINEAR, factor=8)
    assert a == 1.0 and w[5].item() == pytest.approx(plain[5] / 8, rel=1e-14)
    w, a = fa.fa_rope_freqs(R, scaling=fa.FA_ROPE_BASE, factor=8)
    b = base * 8 ** (R / (R - 2))
    assert w[5].item() == pytest.approx(b ** (-10 / R), rel=1e-13)
    # the lowest frequency is divided by the factor, the highest kept
    assert w[-1].item() == pytest.approx(plain[-1] / 8, rel=1e-12) and w[0] == 1.0
    w, a = fa.fa_rope_freqs(R, scaling=fa.FA_ROPE_BY_PARTS, factor=8, trained_len=4096)
    assert a == pytest.approx(0.1 * math.log(8) + 1, rel=1e-6)
    for i in range(R // 2):
        turns = 4096 * plain[i] / (2 * math.pi)
        g = min(1.0, max(0.0, (turns - 1) / 31))
        assert w[i].item() == pytest.approx(plain[i] * (g + (1 - g) / 8), rel=1e-13)
    assert w[0] == 1.0 and w[-1].item() == pytest.approx(plain[-1] / 8, rel=1e-14)


@pytest.mark.parametrize("kw", [dict(rot_dim=0), dict(rot_dim=3), dict(rot_dim=514),
                                dict(rot_dim=64, base=0.0), dict(rot_dim=64, base=math.nan),
                                dict(rot_dim=64, scaling=4), dict(rot_dim=64, scaling=-1),
                                dict(rot_dim=64, scaling=1, factor=0.5),
                                dict(rot_dim=64, scaling=1, factor=math.inf),
                                dict(rot_dim=2, scaling=2, factor=2.0),
                                dict(rot_dim=64, scaling=3, factor=2.0),
                                dict(rot_dim=64, scaling=3, factor=2.0, trained_len=4096,
                                     fast=1.0, slow=1.0)], ids=str)
def test_frequency_refusals(L, kw):
    with pytest.raises(fa.FaError) as e:
        fa.fa_rope_freqs(**kw)
    assert e.value.status == INVALID


# ------------------------------------------------------------------ fa_rope

def rope(L, **kw):
    a = dict(x=A, y=A, pos=A, fr=A, T=4, H=2, d=64, rot=64, xt=128, xh=64, yt=128, yh=64, style=0,
             amp=1.0, inv=0, dtype=0)
    a.update(kw)
    return L.fa_rope(a["x"], a["y"], a["pos"], a["fr"], a["T"], a["H"], a["d"], a["rot"], a["xt"],
                     a["xh"], a["yt"], a["yh"], a["style"], a["amp"], a["inv"], a["dtype"], None)


@pytest.mark.parametrize("kw,want", [
    (dict(T=0, x=None), OK), (dict(T=-1), INVALID), (dict(H=0), INVALID), (dict(d=1), INVALID),
    (dict(d=514, xh=514, yh=514), INVALID), (dict(d=63, rot=62), UNSUPPORTED), (dict(rot=0), INVALID), (dict(rot=63), INVALID),
    (dict(rot=66), INVALID), (dict(style=2), INVALID), (dict(amp=math.inf), INVALID),
    (dict(dtype=3), UNSUPPORTED), (dict(x=None), INVALID), (dict(pos=None), INVALID),
    (dict(fr=None), INVALID), (dict(x=A + 1), INVALID), (dict(dtype=2, y=A + 2), INVALID),
    (dict(fr=A + 4), INVALID), (dict(pos=A + 2), INVALID), (dict(xh=60), INVALID),
    (dict(xt=256), INVALID),                 # in place with other steps
    (dict(y=2 * A, yt=100), INVALID),        # rows of y overlap
    (dict(y=2 * A, yt=-128), INVALID)], ids=str)
def test_rope_refusals(L, kw, want):
    assert rope(L, **kw) == want


# ------------------------------------------------------------------ structs

def fill(cls, base, kw):
    a = dict(base, **kw)
    return cls(*[a[f] for f, _ in cls._fields_])


APPEND = dict(q=A, k=A, v=A, q_out=A, k_pages=A, v_pages=A, block_table=A, ctx_lens=A,
              cu_seqlens=A, freqs=A, q_token=256, k_token=128, v_token=128, q_out_token=256, T=5,
              B=2, H=4, Hkv=2, d=64, rot_dim=64, page_size=16, max_pages_per_seq=4, num_pages=8,
              style=0, amplitude=1.0, dtype=0)


@pytest.mark.parametrize("kw,want", [
    (dict(T=0, q=None), OK), (dict(T=-1), INVALID), (dict(B=0), INVALID), (dict(d=96), UNSUPPORTED),
    (dict(dtype=2), UNSUPPORTED), (dict(page_size=24), UNSUPPORTED), (dict(rot_dim=66), INVALID),
    (dict(rot_dim=7), INVALID), (dict(style=5), INVALID), (dict(amplitude=math.nan), INVALID),
    (dict(q=None), INVALID), (dict(k=A + 8), INVALID), (dict(v_token=120), INVALID),
    (dict(k_token=132), INVALID), (dict(q_out=A, q_out_token=264), INVALID),
    (dict(k_pages=None), INVALID), (dict(v_pages=A + 8), INVALID), (dict(block_table=None), INVALID),
    (dict(ctx_lens=A + 2), INVALID), (dict(freqs=A + 4), INVALID), (dict(num_pages=0), INVALID),
    (dict(page_size=4096, max_pages_per_seq=1 << 20), INVALID)], ids=str)
def test_append_refusals(L, kw, want):
    assert L.fa_rope_append(ctypes.byref(fill(fa.RopeAppendParams, APPEND, kw)), None) == want


VARLEN = dict(q=A, k=A, v=A, o=A, lse=A, q_token=256, k_token=128, v_token=128, o_token=256,
              cu_seqlens_q=A, cu_seqlens_k=A, B=2, H=4, Hkv=2, d=64, total_q=10, total_k=12,
              scale=0.125, mask_mode=1, window=0, n_global=0, dtype=0, workspace=A,
              workspace_bytes=1 << 40, timeout_us=0)
SHARED = [
    (dict(B=0), INVALID), (dict(H=3), INVALID), (dict(Hkv=0), INVALID), (dict(d=96), UNSUPPORTED),
    (dict(H=258, q_token=258 * 64, o_token=258 * 64), UNSUPPORTED), (dict(dtype=2), UNSUPPORTED),
    (dict(scale=math.nan), INVALID), (dict(scale=0.0), INVALID), (dict(scale=-0.1), INVALID), (dict(mask_mode=6), INVALID),
    (dict(mask_mode=5), UNSUPPORTED), (dict(mask_mode=2, window=0), INVALID),
    (dict(mask_mode=2, window=1, n_global=-1), INVALID), (dict(mask_mode=3, window=-1), INVALID),
    (dict(mask_mode=4, n_global=-1), INVALID), (dict(total_q=-1), INVALID),
    (dict(total_q=(1 << 30) + 1), INVALID), (dict(q=None), INVALID), (dict(o=A + 8), INVALID),
    (dict(q_token=252), INVALID), (dict(q_token=248), INVALID), (dict(o_token=1), INVALID),
    (dict(cu_seqlens_q=None), INVALID), (dict(cu_seqlens_q=A + 2), INVALID),
    (dict(lse=A + 2), INVALID), (dict(workspace=None), INVALID), (dict(workspace=A + 8), INVALID),
    (dict(workspace_bytes=64), INVALID)]


@pytest.mark.parametrize("kw,want", SHARED + [
    (dict(total_q=0, q=None, o=None, workspace=None), OK), (dict(total_k=-1), INVALID),
    (dict(k=None), INVALID), (dict(v=A + 8), INVALID), (dict(v_token=100), INVALID),
    (dict(cu_seqlens_k=None), INVALID)], ids=str)
def test_varlen_refusals(L, kw, want):
    assert L.fa_fwd_varlen(ctypes.byref(fill(fa.VarlenParams, VARLEN, kw)), None) == want


PAGED = dict(q=A, k_pages=A, v_pages=A, block_table=A, ctx_lens=A, cu_seqlens_q=A, o=A, lse=A,
             q_token=256, o_token=256, B=2, H=4, Hkv=2, d=64, total_q=10, max_q=8, page_size=16,
             max_pages_per_seq=4, num_pages=8, scale=0.125, mask_mode=1, window=0, n_global=0,
             dtype=0, workspace=A, workspace_bytes=1 << 40, timeout_us=0)


@pytest.mark.parametrize("kw,want", SHARED + [
    (dict(total_q=0, q=None, o=None, workspace=None), OK), (dict(max_q=-1), INVALID),
    (dict(page_size=24), UNSUPPORTED), (dict(page_size=8192), UNSUPPORTED),
    (dict(max_pages_per_seq=0), INVALID), (dict(num_pages=0), INVALID),
    (dict(k_pages=None), INVALID), (dict(v_pages=A + 8), INVALID),
    (dict(block_table=None), INVALID), (dict(ctx_lens=A + 1), INVALID),
    (dict(page_size=4096, max_pages_per_seq=1 << 20), INVALID),
    (dict(page_size=4096, max_pages_per_seq=1 << 18, H=128, Hkv=128, q_token=8192, o_token=8192,
          max_q=1), INVALID),
    (dict(page_size=4096, max_pages_per_seq=1 << 18, H=64, Hkv=64, q_token=4096, o_token=4096,
          max_q=1, B=1 << 9), INVALID)], ids=str)
def test_paged_varlen_refusals(L, kw, want):
    p = fill(fa.PagedVarlenParams, PAGED, kw)
    assert L.fa_fwd_paged_varlen(ctypes.byref(p), None) == want


GRADS = dict(dout=A, dq=A, dk=A, dv=A, dout_token=256, dq_token=256, dk_token=128, dv_token=128)


@pytest.mark.parametrize("kw,gkw,want", [(kw, {}, w) for kw, w in SHARED] + [
    ({}, dict(dout=None), INVALID), ({}, dict(dq=A + 8), INVALID), ({}, dict(dk=None), INVALID),
    ({}, dict(dv_token=100), INVALID), ({}, dict(dq_token=252), INVALID),
    (dict(lse=None), {}, INVALID),
    (dict(total_q=0, total_k=0, q=None, k=None, workspace=None), {}, OK)], ids=str)
def test_bwd_varlen_refusals(L, kw, gkw, want):
    p, g = fill(fa.VarlenParams, VARLEN, kw), fill(fa.VarlenGrads, GRADS, gkw)
    assert L.fa_bwd_varlen(ctypes.byref(p), ctypes.byref(g), None) == want
    assert L.fa_bwd_varlen(ctypes.byref(p), None, None) == INVALID


def test_null_params(L):
    for name in ("fa_rope_append", "fa_fwd_varlen", "fa_fwd_paged_varlen"):
        assert getattr(L, name)(None, None) == INVALID


def test_workspace_sizes_of_bad_shapes(L):
    assert fa.fa_varlen_workspace_size(0, 4, 2, 8, 8, 64) == 0
    assert fa.fa_varlen_workspace_size(1, 4, 3, 8, 8, 64) == 0
    assert fa.fa_varlen_workspace_size(1, 4, 2, 8, 8, 64) > 0
    assert fa.fa_paged_varlen_workspace_size(1, 4, 2, 8, 1, 4, 16, 64) > 0


def test_struct_layouts_match_header(tmp_path):
    import os
    import subprocess
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    structs = {"fa_rope_append_params": fa.RopeAppendParams, "fa_varlen_params": fa.VarlenParams,
               "fa_varlen_grads": fa.VarlenGrads,
               "fa_paged_varlen_params": fa.PagedVarlenParams}
    lines = ["#include <stdio.h>", "#include <stddef.h>", '#include "fa.h"', "int main(void){"]
    for st, cls in structs.items():
        lines.append(f'printf("{st} %zu\\n", sizeof({st}));')
        for f, _ in cls._fields_:
            lines.append(f'printf("{st}.{f} %zu\\n", offsetof({st}, {f}));')
    src = tmp_path / "layout.c"
    src.write_text("\n".join(lines + ["return 0;}"]))
    exe = tmp_path / "layout"
    subprocess.run(["gcc", "-I", os.path.join(root, "include"), str(src), "-o", str(exe)],
                   check=True)
    got = dict(x.split() for x in subprocess.run([str(exe)], capture_output=True, text=True,
                                                 check=True).stdout.splitlines())
    for st, cls in structs.items():
        assert int(got[st]) == ctypes.sizeof(cls)
        for f, _ in cls._fields_:
            assert int(got[f"{st}.{f}"]) == getattr(cls, f).offset, f


def test_cpu_tensors_are_refused():
    x = torch.zeros(2, 2, 64, dtype=torch.float16)
    with pytest.raises(fa.FaError) as e:
        fa.fa_rope(x, x, torch.zeros(2, dtype=torch.int32), torch.zeros(32, dtype=torch.float64))
    assert e.value.status == INVALID


# ------------------------------------------------------------------ the binding's own refusals

@pytest.mark.parametrize("cls,pack", [(fa.RopeAppendParams, "append"), (fa.VarlenParams, "varlen"),
                                      (fa.VarlenGrads, "grads"), (fa.PagedVarlenParams, "paged")])
def test_values_that_do_not_fit_their_field_are_refused(cls, pack):
    pack = getattr(fa, "_pack_" + pack)
    good = [1.0 if t is ctypes.c_float else 1 for _, t in cls._fields_]
    assert bytes(pack(*good)) == bytes(cls(*good))[:len(pack(*good))]
    for i, (name, t) in enumerate(cls._fields_):
        # (a float out of range becomes an infinity, which the library refuses)
        for bad in (2 ** 64, -2 ** 64, None) if t is not ctypes.c_float else (None,):
            with pytest.raises(fa.FaError, match=name) as e:
                pack(*(good[:i] + [bad] + good[i + 1:]))
            assert e.value.status == INVALID
        if t is ctypes.c_int:
            for bad in (2 ** 31, -2 ** 31 - 1, 2 ** 32 + 1, 0.5):
                with pytest.raises(fa.FaError, match=name):
                    pack(*(good[:i] + [bad] + good[i + 1:]))


@pytest.mark.parametrize("name,n", [("fa_varlen_workspace_size", 6),
                                    ("fa_bwd_varlen_workspace_size", 6),
                                    ("fa_paged_varlen_workspace_size", 8)])
def test_workspace_sizes_refuse_what_an_int_does_not_hold(L, name, n):
    size = getattr(fa, name)
    good = dict([("B", 1), ("H", 4), ("Hkv", 2), ("total_q", 8)] +
                ([("total_k", 8)] if n == 6 else [("max_q", 8), ("max_pages_per_seq", 2),
                                                  ("page_size", 16)]) + [("d", 64)])
    assert size(**good) > 0
    for key in good:
        for bad in (2 ** 32 + good[key], 2 ** 31, -2 ** 31 - 1, 1.5, None):
            with pytest.raises(fa.FaError, match=key):
                size(**dict(good, **{key: bad}))


def test_frequencies_refuse_what_an_int_does_not_hold(L):
    for kw in (dict(rot_dim=2 ** 32 + 64), dict(rot_dim=2 ** 31 - 2), dict(rot_dim=64.0),
               dict(rot_dim=64, scaling=2 ** 32),
               dict(rot_dim=64, scaling=3, factor=2.0, trained_len=2 ** 32 + 4096)):
        with pytest.raises(fa.FaError) as e:
            fa.fa_rope_freqs(**kw)
        assert e.value.status == INVALID
