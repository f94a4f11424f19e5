"""Attention of new tokens over an 8-bit cache, of trees of drafted tokens over either cache, and the
calls around them run together, against the definition in 64 bits (_packed.py has the tolerances:
an 8-bit cache's values are exact in both kernels' products, so they are the 16-bit calls')."""
import pytest
import torch

import _cache8 as c8
import _packed as ref
import tiled_attention_06_gb300 as fa

pytestmark = pytest.mark.gpu
BF, HF = torch.bfloat16, torch.float16
NONE, CAUSAL, WINDOW = fa.FA_MASK_NONE, fa.FA_MASK_CAUSAL, fa.FA_MASK_CAUSAL_WINDOW
BAND, PREFIX, TREE = fa.FA_MASK_BAND, fa.FA_MASK_PREFIX_LM, fa.FA_MASK_TREE


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


class Call:
    """Queries, cache, outputs and workspace of one call."""

    def __init__(self, lens, ctx, H, Hkv, d, page, dtype, bits=8, mask=CAUSAL, window=0, n_global=0,
                 words=None, blank=(), seed=0, q=None, rows=None, max_q=None):
        self.lens, self.ctx, self.dtype, self.d = lens, ctx, dtype, d
        T = sum(lens)
        self.T, self.H, self.Hkv = T, H, Hkv
        g = torch.Generator().manual_seed(seed + 100)
        wide = torch.randn(T + 2, H + 1, d, generator=g) if q is None else q
        self.wide = wide.to(dtype)
        self.q = self.wide[:, :H]
        self.cache = c8.Cache(ctx, Hkv, d, page, seed, bits, dtype, rows)
        self.scale = d ** -0.5
        self.mask = dict(mask=mask, window=window, n_global=n_global)
        self.tree = None
        if mask == TREE:
            words = words or -(-max(max(lens), 1) // 32)
            self.tree = c8.trees(lens, words, seed, blank)
        self.max_q = max(lens) if max_q is None else max_q
        self.qd = self.wide.cuda()[:, :H]
        (self.k, self.v, self.table), self.kw = self.cache.cuda()
        if self.tree is not None:
            self.kw["tree"] = self.tree.cuda()
        else:
            self.kw.update(mask_mode=mask, window=window, n_global=n_global)
        self.ctx_d, self.cu = i32(ctx), i32(ref.starts(lens))
        self.o = torch.full((T + 2, H, d), 7.0, dtype=dtype, device="cuda")
        self.lse = torch.full((T + 2, H), 7.0, device="cuda")
        self.ws = torch.full((fa.fa_paged_varlen_workspace_size(
            len(lens), H, Hkv, T + 2, self.max_q, self.table.shape[1], page, d),), 255,
            dtype=torch.uint8, device="cuda")

    def run(self, stream=None):
        fa.fa_fwd_paged_varlen_ex(self.qd, self.k, self.v, self.table, self.ctx_d, self.cu, self.max_q,
                                  self.o, self.lse, self.scale, self.ws, stream=stream, **self.kw)

    def run_and_check(self):
        self.run()
        self.check()

    def check(self, what=""):
        torch.cuda.synchronize()
        assert fa.fa_get_device_status() == fa.FA_OK
        want = c8.attention(self.q[:self.T], self.cache, self.ctx, self.lens, self.scale,
                            tree=self.tree, **self.mask)
        ref.check_forward(self.o, self.lse, want, self.dtype, self.T, what)
        assert (self.o[self.T:] == 7).all() and (self.lse[self.T:] == 7).all()


SHAPES = [  # lengths, keys, H, Hkv, d, page, dtype
    ([1], [1], 1, 1, 64, 16, BF),
    ([1, 1, 1, 1], [1, 64, 65, 700], 8, 2, 128, 64, HF),
    ([1, 0, 1], [0, 5, 2049], 16, 1, 128, 16, BF),       # no keys, no tokens
    ([4, 3, 1], [4, 300, 129], 8, 2, 64, 48, HF),        # few rows, pages that end inside a tile
    ([2, 2], [3000, 17], 6, 3, 128, 256, BF),
    ([16], [900], 1, 1, 64, 4096, BF),
    ([17, 1, 5], [17, 128, 600], 4, 4, 128, 64, BF),     # 128-row tiles
    ([40, 0, 130], [40, 3, 1000], 8, 2, 128, 16, HF),
    ([33], [1025], 5, 1, 64, 128, BF),
    ([300, 1, 64], [700, 1500, 64], 12, 4, 64, 80, HF),
    ([7, 9], [5, 9], 8, 2, 128, 32, BF),                 # more tokens than keys
    ([1, 2], [513, 200], 128, 1, 64, 64, BF),
]
MASKS = [(CAUSAL, 0, 0), (NONE, 0, 0), (WINDOW, 70, 3), (BAND, 20, 0), (PREFIX, 0, 90)]


@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("mask", MASKS, ids=str)
def test_positional_masks_over_8_bits(shape, mask):
    c = Call(*shape, mask=mask[0], window=mask[1], n_global=mask[2], seed=len(shape[0]))
    c.run()
    c.check()


@pytest.mark.parametrize("bits", [8, 16])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_trees(shape, bits):
    c = Call(*shape, bits=bits, mask=TREE, seed=3)
    c.run()
    c.check()


LONG = [  # items cut into pieces for the SMs, among them sequences without keys or tokens
    ([64], [6000], 8, 2, 128, 64, BF),
    ([40, 0, 3, 64, 20], [5000, 4000, 0, 9000, 20], 4, 4, 64, 128, HF),
    ([33, 200], [3000, 7000], 2, 1, 128, 16, HF),
]


@pytest.mark.parametrize("shape", LONG, ids=str)
@pytest.mark.parametrize("mask", MASKS + [(WINDOW, 2500, 300), (BAND, 1500, 0)], ids=str)
def test_pieces_over_8_bits(shape, mask):
    test_positional_masks_over_8_bits(shape, mask)


@pytest.mark.parametrize("bits", [8, 16])
@pytest.mark.parametrize("shape", LONG, ids=str)
def test_pieces_with_trees(shape, bits):
    test_trees(shape, bits)


@pytest.mark.parametrize("mask,bits", [(CAUSAL, 8), (WINDOW, 8), (TREE, 8), (TREE, 16)])
@pytest.mark.parametrize("lens", [[1, 2, 0], [1, 17, 0]])
def test_many_short_sequences(lens, mask, bits):
    """More sequences than threads, few rows and tiles."""
    Call(lens * 400, [3, 40, 0] * 400, 2, 1, 64, 16, BF, bits=bits, mask=mask,
         window=2 if mask == WINDOW else 0, n_global=1 if mask == WINDOW else 0).run_and_check()


@pytest.mark.parametrize("bits", [8, 16])
@pytest.mark.parametrize("lens,ctx", [([3, 2], [3, 2]), ([40, 2], [40, 80])])
def test_tokens_that_see_nothing(lens, ctx, bits):
    """No earlier key and no bit: o = 0 and lse = -inf. More words than the chunks need."""
    c = Call(lens, ctx, 4, 2, 64, 16, HF, bits=bits, mask=TREE, words=5, blank=(0, 2))
    c.run()
    c.check()
    assert (c.o[0] == 0).all() and c.lse[0].isneginf().all()


@pytest.mark.parametrize("bits", [8, 16])
def test_a_chain_is_the_causal_mask(bits):
    for lens, ctx in (([5, 3], [200, 70]), ([70, 33], [300, 33])):
        c = Call(lens, ctx, 4, 2, 128, 64, BF, bits=bits, mask=TREE)
        rows = [(2 << j) - 1 for n in lens for j in range(n)] + [0, 0]
        words = c.tree.shape[1]
        c.kw["tree"].copy_(torch.tensor([[(r >> 32 * w) & 0xffffffff for w in range(words)]
                                         for r in rows]).to(torch.int32))
        c.run()
        tree = c.o.clone(), c.lse.clone()
        del c.kw["tree"]
        c.run()
        torch.cuda.synchronize()
        assert torch.equal(tree[0], c.o) and torch.equal(tree[1], c.lse)


def test_16_bits_without_a_tree_is_the_plain_call():
    for lens, ctx in (([1, 2], [300, 70]), ([70, 33], [300, 33])):
        c = Call(lens, ctx, 4, 2, 128, 64, BF, bits=16)
        c.run()
        o, lse = c.o.clone(), c.lse.clone()
        fa.fa_fwd_paged_varlen(c.qd, c.k, c.v, c.table, c.ctx_d, c.cu, c.max_q, c.o, c.lse, c.scale,
                               c.ws)
        torch.cuda.synchronize()
        assert torch.equal(o, c.o) and torch.equal(lse, c.lse)


# ------------------------------------------------------------------------------ numbers

def uneven(low, high):
    """Rows whose powers of two are far apart."""
    def make(*shape):
        g = torch.Generator().manual_seed(7)
        return torch.randn(*shape, 64, generator=g) * torch.exp2(
            torch.randint(low, high + 1, (*shape, 1), generator=g).float())
    return make


@pytest.mark.parametrize("lens,ctx", [([1, 2], [400, 130]), ([50], [500])])
@pytest.mark.parametrize("dtype,low,high", [(BF, -60, 40), (HF, -14, 6), (BF, 10, 60)])
def test_rows_of_very_different_sizes(lens, ctx, dtype, low, high):
    """K and V rows from 2^low to 2^high; queries small enough for scores below 100."""
    T = sum(lens)
    q = torch.randn(T + 2, 3, 64, generator=torch.Generator().manual_seed(1)) * 2.0 ** (-max(high, 0))
    c = Call(lens, ctx, 2, 1, 64, 16, dtype, q=q, rows=uneven(low, high))
    c.run()
    c.check()


@pytest.mark.parametrize("lens,ctx", [([1, 2], [400, 130]), ([50], [500])])
@pytest.mark.parametrize("size", [1e-34, 1e-30, 1e-3, 1e4, 1e30, 1e37])
def test_queries_of_any_size(lens, ctx, size):
    """bf16 queries far outside FP16's range, keys that bring the scores back."""
    T = sum(lens)
    q = torch.randn(T + 2, 3, 64, generator=torch.Generator().manual_seed(1)) * size
    g = torch.Generator().manual_seed(2)
    c = Call(lens, ctx, 2, 1, 64, 16, BF, q=q,
             rows=lambda *s: torch.randn(*s, 64, generator=g) / size)
    c.run()
    c.check()


@pytest.mark.parametrize("lens,ctx", [([1, 2], [400, 130]), ([50, 3], [500, 90])])
def test_nan_rows(lens, ctx):
    """A key that could not be scaled: NaN for the queries that see it, the others keep theirs."""
    for which in (0, 1):
        c = Call(lens, ctx, 2, 1, 64, 16, BF)
        at = ctx[0] - 2
        page = c.cache.table[0, at // 16].item()
        (c.k if which == 0 else c.v).view(torch.uint8)[page, 0, at % 16] = 0
        c.kw["k_scales" if which == 0 else "v_scales"].view(torch.uint8)[page, 0, at % 16] = 255
        c.run()
        torch.cuda.synchronize()
        sees = [i for i in range(lens[0]) if ctx[0] - lens[0] + i >= at]
        assert c.o[sees].isnan().all()
        if which == 0:
            assert c.lse[sees].isnan().all()
            hidden = [i for i in range(lens[0]) if i not in sees]
            assert torch.isfinite(c.o[hidden].float()).all()
        rest = slice(lens[0], c.T)
        want = c8.attention(c.q[:c.T], c.cache, ctx, lens, c.scale, CAUSAL)
        err = (c.o[rest].double().cpu() - want[0][rest]).abs().amax(-1)
        assert (err <= 2 * 2.0 ** -8 * want[2][rest] + 2.0 ** -17 * (1 + want[2][rest])).all()


# ------------------------------------------------------------------------------ how it is called

def test_bad_pages_are_reported():
    for lens, ctx in (([1, 2], [40, 30]), ([40, 2], [60, 30])):
        c = Call(lens, ctx, 2, 1, 64, 16, BF)
        c.table[0, 1] = 999
        c.run()
        torch.cuda.synchronize()
        assert fa.fa_get_device_status() == fa.FA_ERR_BAD_PAGE
        want = c8.attention(c.q[:c.T], c.cache, ctx, lens, c.scale, CAUSAL)
        got = c.o[lens[0]:c.T].double().cpu()
        assert ((got - want[0][lens[0]:]).abs().amax(-1) <= 2.0 ** -6 * want[2][lens[0]:]).all()


@pytest.mark.parametrize("lens,ctx", [([2, 1], [300, 70]), ([64, 40], [400, 90])])
@pytest.mark.parametrize("bits", [8, 16])
def test_captured_call_follows_lengths_and_trees(lens, ctx, bits):
    c = Call(lens, ctx, 4, 2, 64, 64, HF, bits=bits, mask=TREE, seed=2)
    c.run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.run()
    c.lens, c.ctx = [lens[0] - 1, lens[1]], [ctx[0] - 30, ctx[1] - 1]
    c.T = sum(c.lens)
    c.cu.copy_(i32(ref.starts(c.lens)))
    c.ctx_d.copy_(i32(c.ctx))
    c.tree = c8.trees(c.lens, c.tree.shape[1], seed=9)
    c.kw["tree"][:c.T + 2].copy_(c.tree)
    c.o.fill_(7)
    c.lse.fill_(7)
    c.ws.fill_(255)
    graph.replay()
    c.check()


def test_two_streams_with_their_own_workspaces():
    calls = [Call([1, 3], [2000, 700], 8, 2, 128, 64, BF, seed=i) for i in range(2)] + \
        [Call([90], [1500], 8, 2, 128, 64, BF, seed=4, bits=b, mask=TREE) for b in (8, 16)]
    streams = [torch.cuda.Stream() for _ in calls]
    torch.cuda.synchronize()
    for _ in range(3):
        for c, s in zip(calls, streams):
            c.run(stream=s)
    for c in calls:
        c.check()


def test_the_same_bits_on_every_run():
    for c in (Call([1] * 5, [3000, 1, 900, 64, 2222], 8, 2, 128, 64, HF),
              Call([200, 31], [1500, 800], 8, 2, 128, 64, BF, mask=TREE)):
        c.run()
        o, lse = c.o.clone(), c.lse.clone()
        c.ws.fill_(255)
        c.run()
        torch.cuda.synchronize()
        assert torch.equal(o, c.o) and torch.equal(lse, c.lse)


def test_far_pages_of_a_large_pool():
    """Rows of the pool beyond 2^31 bytes."""
    d, page, Hkv = 128, 4096, 8
    P = 600  # 600 * 8 * 4096 * 128 bytes = 2.5 GB a pool
    c = Call([1, 40], [100, 300], 8, 8, d, page, BF)
    k = torch.zeros(P, Hkv, page, d, dtype=torch.uint8, device="cuda")
    v = torch.zeros_like(k)
    ks, vs = (torch.zeros(P, Hkv, page, dtype=torch.uint8, device="cuda") for _ in range(2))
    n = c.k.shape[0]
    for big, small in ((k, c.k), (v, c.v), (ks, c.kw["k_scales"]), (vs, c.kw["v_scales"])):
        big[P - n:].copy_(small.view(torch.uint8))
    c.k, c.v, c.kw["k_scales"], c.kw["v_scales"] = k, v, ks, vs
    c.table.add_(torch.where(c.table >= 0, P - n, 0).to(torch.int32))
    for few in (True, False):
        c.max_q = 40
        if few:
            c.cu.copy_(i32([0, 1, 1]))
            c.max_q = 1
        else:
            c.cu.copy_(i32([0, 1, 41]))
        c.ws = torch.empty(fa.fa_paged_varlen_workspace_size(2, 8, 8, c.o.shape[0], c.max_q,
                                                             c.table.shape[1], page, d),
                           dtype=torch.uint8, device="cuda")
        c.run()
    c.check()


# ------------------------------------------------------------------------------ run together

@pytest.mark.parametrize("dtype", [BF, HF])
def test_a_layer_with_drafted_trees(dtype):
    """What a serving step does: norm and rotate the drafted tokens by their depths, write them into
    the 8-bit cache, attend to it under the tree's mask, and read the chunks back; the reference
    follows the cache's own bytes. Then one accepted token more, alone."""
    H, Hkv, d, page, axes = 8, 2, 128, 64, 3
    lens, before = [5, 12, 1], [300, 0, 63]
    ctx = [a + b for a, b in zip(lens, before)]
    T = sum(lens)
    c = Call(lens, ctx, H, Hkv, d, page, dtype, mask=TREE, seed=11)
    g = torch.Generator().manual_seed(3)
    qkv = torch.randn(T + 2, H + 2 * Hkv, d, generator=g).to(dtype)
    dev = qkv.cuda()
    depth = torch.zeros(T + 2, dtype=torch.int64)
    for b, (n, s) in enumerate(zip(lens, before)):
        for i in range(n):
            row = int(c.tree[sum(lens[:b]) + i, 0]) & ((1 << n) - 1)
            depth[sum(lens[:b]) + i] = s + bin(row).count("1") - 1
    pos = depth.expand(axes, T + 2).contiguous()
    pos[1:] += torch.randint(0, 30, (2, T + 2), generator=g)
    axis = fa.fa_rope_axes([16, 24, 24])
    freqs = fa.fa_rope_freqs(d)[0]
    w = [(1 + 0.1 * torch.randn(d, generator=g)).to(dtype) for _ in range(2)]
    q_rot = torch.zeros(T + 2, H, d, dtype=dtype, device="cuda")
    fa.fa_norm_rope_append(dev[:, :H], dev[:, H:H + Hkv], dev[:, H + Hkv:], q_rot, c.k, c.v, c.table,
                           i32(before), c.cu, freqs.cuda(), positions=pos.to(torch.int32).cuda(),
                           pair_axis=axis.cuda(), q_weight=w[0].cuda(), k_weight=w[1].cuda(),
                           norm=fa.FA_NORM_RMS, k_scales=c.kw["k_scales"], v_scales=c.kw["v_scales"])
    c.qd = q_rot
    c.run()
    rows = [torch.zeros(T + 2, Hkv, d, dtype=dtype, device="cuda") for _ in range(2)]
    fa.fa_kv_read(c.k, c.v, c.kw["k_scales"], c.kw["v_scales"], c.table, i32(before), c.cu, *rows)
    torch.cuda.synchronize()
    args = (pos[:, :T], axis, freqs, d, True)
    y, bound = c8.norm_rope(qkv[:T, :H], w[0], 1e-6, *args)
    c8.check(q_rot[:T], y, bound, dtype, "q")
    c.cache.pages = [x.view(torch.uint8).cpu() for x in (c.k, c.v)]
    c.cache.scales = [c.kw[n].view(torch.uint8).cpu() for n in ("k_scales", "v_scales")]
    at = 0
    for b, (n, m) in enumerate(zip(lens, ctx)):
        for got, x in zip(rows, c.cache.rows(b, m)):
            assert torch.equal(got[at:at + n].cpu(), x[m - n:].to(dtype))
        at += n
    k, kb = c8.norm_rope(qkv[:T, H:H + Hkv], w[1], 1e-6, *args)
    # what is read back is within half a step of 8 bits (2^-4) of the row, and its own rounding
    err = (rows[0][:T].double().cpu() - k).abs()
    assert (err <= 2.0 ** -4 * k.abs() + 2.0 ** -9 * k.abs().amax(-1, keepdim=True) + kb).all()
    c.q = q_rot.cpu()
    c.check("drafts")
    # one token more for every sequence, by its place
    one = Call([1, 1, 1], [m + 1 for m in ctx], H, Hkv, d, page, dtype, seed=11)
    one.k, one.v, one.table = c.k, c.v, c.table
    one.kw.update(k_scales=c.kw["k_scales"], v_scales=c.kw["v_scales"])
    if any(-(-m // page) > (t >= 0).sum() for m, t in zip(one.ctx, c.cache.table)):
        one.table[2, 1] = c.k.shape[0] - 1 if not (c.table == c.k.shape[0] - 1).any() else \
            [p for p in range(c.k.shape[0]) if not (c.table == p).any()][0]
    new = torch.randn(5, H + 2 * Hkv, d, generator=g).to(dtype).cuda()
    out = torch.zeros(5, H, d, dtype=dtype, device="cuda")
    fa.fa_norm_rope_append(new[:, :H], new[:, H:H + Hkv], new[:, H + Hkv:], out, one.k, one.v,
                           one.table, i32(ctx), one.cu, freqs.cuda(), q_weight=w[0].cuda(),
                           k_weight=w[1].cuda(), norm=fa.FA_NORM_RMS, k_scales=c.kw["k_scales"],
                           v_scales=c.kw["v_scales"])
    one.qd = out
    one.run()
    torch.cuda.synchronize()
    one.q = out.cpu()
    one.cache.table = one.table.cpu()
    one.cache.pages = [x.view(torch.uint8).cpu() for x in (c.k, c.v)]
    one.cache.scales = [c.kw[n].view(torch.uint8).cpu() for n in ("k_scales", "v_scales")]
    one.check("step")
