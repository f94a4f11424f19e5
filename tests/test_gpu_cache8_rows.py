"""Attention over an 8-bit cache whose rows of V are very different in size: a query's output depends on
the rows that it sees alone, and on each as much as its probability says.

Tolerances as in _packed.py, with the largest row that the query sees. In the second test the bound is of
the terms: each P_j |v_j| is off by one rounding, u of itself (and what FP16 loses below 2^-24 of a
warp's unit, 2^-22 of the largest term for each key; FP32 exponentials 2^-18); O is rounded once more.
"""
import pytest
import torch

import _cache8 as c8
import _packed as ref
import tiled_attention_06_gb300 as fa
from test_gpu_cache8 import Call

pytestmark = pytest.mark.gpu
BF, HF = torch.bfloat16, torch.float16
CAUSAL, WINDOW = fa.FA_MASK_CAUSAL, fa.FA_MASK_CAUSAL_WINDOW
BAND, PREFIX, TREE = fa.FA_MASK_BAND, fa.FA_MASK_PREFIX_LM, fa.FA_MASK_TREE


def lift(c, b, places, by):
    """V's rows at these positions of sequence b times 2^by, in every head."""
    gpu = c.kw["v_scales"].view(torch.uint8)
    for at in places:
        page, slot = c.cache.table[b, at // c.cache.page].item(), at % c.cache.page
        c.cache.scales[1][page, :, slot] += by
        gpu[page, :, slot] += by


def forest(c):
    """Every token sees itself and the keys before the chunk."""
    bits = [1 << j for n in c.lens for j in range(n)] + [0, 0]
    c.tree.copy_(torch.tensor(bits, dtype=torch.int64).to(torch.int32)[:, None])
    c.kw["tree"].copy_(c.tree)


HIDDEN = [  # name, lengths, keys, mask, window, n_global, lifted positions counted from each end
    ("window of one", [1, 1], [40, 700], WINDOW, 1, 0, [-2, -5]),
    ("before the window", [1, 1], [400, 1500], WINDOW, 200, 0, [-201, -210]),
    ("beside global keys", [2, 1], [90, 1500], WINDOW, 40, 3, [4, 5, -70]),
    ("causal", [2, 2], [50, 900], CAUSAL, 0, 0, [-1]),
    ("band", [2, 2], [300, 900], BAND, 20, 0, [-24, -40]),
    ("prefix", [2, 2], [70, 900], PREFIX, 0, 20, [-1]),
    ("siblings", [2, 2], [35, 900], TREE, 0, 0, [-2]),
]


@pytest.mark.parametrize("by", [18, 26, 60])
@pytest.mark.parametrize("H,Hkv,d,dtype", [(2, 1, 64, BF), (8, 2, 128, HF), (7, 1, 128, BF), (5, 1, 64, HF),
                                           (20, 1, 64, BF)], ids=str)
@pytest.mark.parametrize("name,lens,ctx,mask,window,n_global,at", HIDDEN, ids=[h[0] for h in HIDDEN])
def test_hidden_rows_of_v_do_not_matter(name, lens, ctx, mask, window, n_global, at, H, Hkv, d, dtype, by):
    """Up to 8, 16 and more rows (tokens x heads of a group)."""
    c = Call(lens, ctx, H, Hkv, d, 16, dtype, mask=mask, window=window, n_global=n_global, words=1, seed=6)
    if mask == TREE:
        forest(c)
    for b, m in enumerate(ctx):
        lift(c, b, [a % m for a in at], by)
    c.run()
    torch.cuda.synchronize()
    assert fa.fa_get_device_status() == fa.FA_OK
    o, lse, bound = c8.attention(c.q[:c.T], c.cache, ctx, lens, c.scale, tree=c.tree, **c.mask)
    # queries that see a lifted row leave FP16's range, others do not
    rows = (bound < 2.0 ** 12) | (dtype is BF)
    assert (bound < 2.0 ** 12).any()
    got = c.o[:c.T].double().cpu()
    err = (got - o).abs().amax(-1)
    lim = 2 * ref.half_step(dtype) * bound + 2.0 ** -18 * (1 + bound)
    assert (err <= lim)[rows].all(), float((err - lim)[rows].max())
    assert ((c.lse[:c.T].double().cpu() - lse).abs() <= 1e-4).all()


@pytest.mark.parametrize("rows,dtype", [(1, BF), (1, HF), (12, BF), (12, HF), (20, BF)], ids=str)
@pytest.mark.parametrize("by", [-40, 40])
def test_every_row_of_v_counts_by_its_probability(rows, by, dtype):
    """The less probable two thirds of the keys 2^40 times larger, or the most probable one smaller."""
    d, m, n = 64, 300, 1
    g = torch.Generator().manual_seed(8)
    q = 12 * torch.randn(n + 2, rows + 1, d, generator=g)
    q[:] = q[:1, :1]  # one query for every row: the same keys are improbable for all
    c = Call([n], [m], rows, 1, d, 16, dtype, q=q, seed=4)
    k, v = c.cache.rows(0, m)
    s = (c.q[0, 0].double() @ k[:, 0].T * c.scale).sort()
    assert s.values[-1] - s.values[0] > 60
    lift(c, 0, (s.indices[:200] if by > 0 else s.indices[-1:]).tolist(), by)
    c.run()
    torch.cuda.synchronize()
    k, v = c.cache.rows(0, m)
    p, o, _ = ref.head(c.q[0, :1], k[:, 0], v[:, 0], torch.ones(1, m, dtype=torch.bool), c.scale)
    term = p * v[:, 0].abs().amax(-1)
    u = ref.half_step(dtype)
    lim = (u + 2.0 ** -18) * term.sum() + m * 2.0 ** -22 * term.max() + u * o.abs().amax()
    lim += 2.0 ** -25 if dtype is HF else 0.0  # half a step of the smallest FP16 numbers
    err = (c.o[0].double().cpu() - o).abs().amax()
    assert err <= lim, (float(err), float(lim))


@pytest.mark.parametrize("kw", [dict(mask_mode=WINDOW, window=8), dict(mask_mode=BAND, window=8),
                                dict(mask_mode=PREFIX, n_global=4), dict(mask_mode=fa.FA_MASK_NONE),
                                dict(window=8), dict(n_global=4), dict(mask_mode=TREE, window=8),
                                dict(mask_mode=9)], ids=str)
def test_a_tree_takes_no_other_mask(kw):
    c = Call([2], [40], 2, 1, 64, 16, BF, mask=TREE)
    c.kw.update(kw)
    with pytest.raises(fa.FaError) as e:
        c.run()
    assert e.value.status == fa.FA_ERR_INVALID_ARG
    torch.cuda.synchronize()
    assert (c.o == 7).all()
    for mask in (TREE, CAUSAL):  # the tree itself, and the default
        c.kw.update(mask_mode=mask, window=0, n_global=0)
        c.run_and_check()


# ------------------------------------------------------------------------------ far pages, FP16's range

@pytest.mark.parametrize("lens", [[1, 0], [1, 40]], ids=["few rows", "tiles"])
def test_rows_beyond_2_to_the_31_bytes(lens):
    """Either kernel over pages in the last 2.5 GB of the pools; rows that no sequence owns stay."""
    d, page, H, P = 128, 4096, 8, 600
    c = Call(lens, [100, 300], H, H, d, page, BF, seed=2)
    n = c.k.shape[0]
    far = []
    for small in (c.k, c.v, c.kw["k_scales"], c.kw["v_scales"]):
        big = torch.zeros(P, *small.shape[1:], dtype=torch.uint8, device="cuda")
        big[P - n:].copy_(small.view(torch.uint8))
        far.append(big)
    c.k, c.v, c.kw["k_scales"], c.kw["v_scales"] = far
    c.table.add_(torch.where(c.table >= 0, P - n, 0).to(torch.int32))
    c.run()
    c.check()


@pytest.mark.parametrize("lens", [[1, 2], [50, 3]], ids=["few rows", "tiles"])
@pytest.mark.parametrize("which", ["k", "v"])
@pytest.mark.parametrize("by,outside", [(8, False), (24, True)])
def test_values_beyond_fp16(lens, which, by, outside):
    """FP16 calls over rows that FP16 does not hold: few rows take them as they are, tiles as
    infinities, which the queries of that sequence show; other sequences keep theirs."""
    ctx, d = [400, 130], 64
    q = torch.randn(sum(lens) + 2, 3, d, generator=torch.Generator().manual_seed(1))
    q *= 2.0 ** -by if which == "k" else 1.0
    c = Call(lens, ctx, 2, 1, d, 16, HF, q=q, seed=3)
    i = "kv".index(which)
    page = c.cache.table[0, 1].item()
    c.cache.scales[i][page] += by
    c.kw[which + "_scales"].view(torch.uint8)[page] += by
    c.run()
    torch.cuda.synchronize()
    assert fa.fa_get_device_status() == fa.FA_OK
    want = c8.attention(c.q[:c.T], c.cache, ctx, lens, c.scale, CAUSAL)
    got = c.o[:c.T].double().cpu()
    ok = (got - want[0]).abs().amax(-1) <= 2 * 2.0 ** -11 * want[2] + 2.0 ** -18 * (1 + want[2])
    first = slice(0, lens[0])
    assert ok[lens[0]:].all()
    if not outside or (lens[0] < 9 and which == "k"):
        assert ok[first].all()
    elif lens[0] < 9:  # the output itself leaves FP16
        assert got[first][want[0][first].abs() > 2.0 ** 17].isinf().all()
    else:
        assert not torch.isfinite(got[first]).all(-1).any()
