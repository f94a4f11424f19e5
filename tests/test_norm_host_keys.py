"""Without key heads nothing of k is looked at, its weight neither: host checks, no GPU."""
import ctypes

import pytest

import tiled_attention_06_gb300 as fa
from test_norm_host import A, GRADS, L, NORM, OK, fill  # noqa: F401


@pytest.mark.parametrize("kw", [dict(k_weight=A + 1), dict(k_weight=A + 2, weight_dtype=2, dtype=2)], ids=str)
def test_the_weight_of_no_key_heads_is_ignored(L, kw):  # noqa: F811
    kw = dict(kw, T=0, Hkv=0, k=1, k_out=3)
    p = ctypes.byref(fill(fa.NormRopeParams, NORM, kw))
    assert L.fa_norm_rope(p, None) == OK
    none = dict(dq_weight=None, dk_weight=None)
    assert L.fa_norm_rope_bwd(p, ctypes.byref(fill(fa.NormRopeGrads, GRADS, none)), None) == OK
    q = dict(kw, q_weight=A + 1)
    assert L.fa_norm_rope(ctypes.byref(fill(fa.NormRopeParams, NORM, q)), None) == fa.FA_ERR_INVALID_ARG
