"""Packed grouped-head attention through the C ABI against a plain implementation in 64 bits
(tolerances: _packed.py)."""
import math

import pytest
import torch

import tiled_attention_06_gb300 as fa

from _packed import attention, check_forward, starts

pytestmark = pytest.mark.gpu

DT = {"f16": torch.float16, "bf16": torch.bfloat16}
MASKS = {"none": (fa.FA_MASK_NONE, 0, 0), "causal": (fa.FA_MASK_CAUSAL, 0, 0),
         "window": (fa.FA_MASK_CAUSAL_WINDOW, 50, 5), "band": (fa.FA_MASK_BAND, 40, 0),
         "prefix": (fa.FA_MASK_PREFIX_LM, 0, 70)}


@pytest.fixture(scope="module", autouse=True)
def _built():
    from tiled_attention_06_gb300 import build
    build.build()
    fa.lib()


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def forward(q, k, v, cu_q, cu_k, scale, mask=(fa.FA_MASK_CAUSAL, 0, 0), want_lse=True):
    """q, k, v on the GPU; o and lse poisoned first."""
    T, H, d = q.shape
    o = torch.full((T, H, d), float("nan"), dtype=q.dtype, device="cuda")
    lse = torch.full((T, H), float("nan"), device="cuda") if want_lse else None
    ws = torch.empty(max(fa.fa_varlen_workspace_size(len(cu_q) - 1, H, k.shape[1], T, k.shape[0],
                                                     d), 16), dtype=torch.uint8, device="cuda")
    fa.fa_fwd_varlen(q, k, v, o, lse, i32(cu_q), i32(cu_k), scale, ws, *mask)
    assert fa.fa_get_device_status() == fa.FA_OK
    return o, lse


def case(lens_q, lens_k, H, Hkv, d, dtype, seed, pad=0):
    g = torch.Generator().manual_seed(seed)
    q = torch.randn(sum(lens_q) + pad, H, d, generator=g).to(dtype)
    k = torch.randn(sum(lens_k) + pad, Hkv, d, generator=g).to(dtype)
    v = torch.randn(sum(lens_k) + pad, Hkv, d, generator=g).to(dtype)
    return q, k, v, starts(lens_q), starts(lens_k)


LENS = [[1], [1, 1, 1], [0, 5, 0], [128], [129, 1, 127], [17, 300, 64, 2], [640]]


@pytest.mark.parametrize("lens", LENS, ids=str)
@pytest.mark.parametrize("H,Hkv,d,dt", [(4, 4, 64, "f16"), (8, 2, 128, "bf16"),
                                        (7, 1, 128, "f16"), (6, 2, 64, "bf16")])
@pytest.mark.parametrize("mask", list(MASKS))
def test_self_attention(lens, H, Hkv, d, dt, mask):
    q, k, v, cu, _ = case(lens, lens, H, Hkv, d, DT[dt], seed=sum(lens) + H, pad=2)
    scale = 1 / math.sqrt(d)
    o, lse = forward(q.cuda(), k.cuda(), v.cuda(), cu, cu, scale, MASKS[mask])
    T = sum(lens)
    check_forward(o, lse, attention(q, k, v, cu, cu, scale, *MASKS[mask]), DT[dt], T,
                  f"{lens} {mask}")
    assert o[T:].isnan().all() and lse[T:].isnan().all()  # rows behind the last sequence


@pytest.mark.parametrize("lens_q,lens_k", [([3, 200, 1], [200, 3, 0]), ([1, 1], [1000, 129]),
                                           ([5], [4099]), ([130, 0, 2], [0, 7, 260])], ids=str)
@pytest.mark.parametrize("G", [1, 5])
@pytest.mark.parametrize("mask", list(MASKS))
def test_other_keys_than_queries(lens_q, lens_k, G, mask):
    """Cross attention, long contexts (split over the SMs), queries without any key."""
    H, Hkv, d = 2 * G, 2, 128
    q, k, v, cu_q, cu_k = case(lens_q, lens_k, H, Hkv, d, torch.bfloat16, seed=G)
    scale = 1 / math.sqrt(d)
    o, lse = forward(q.cuda(), k.cuda(), v.cuda(), cu_q, cu_k, scale, MASKS[mask])
    check_forward(o, lse, attention(q, k, v, cu_q, cu_k, scale, *MASKS[mask]), torch.bfloat16,
                  sum(lens_q), f"{lens_q} {lens_k} {mask}")


@pytest.mark.parametrize("mask", [(fa.FA_MASK_CAUSAL_WINDOW, 2 ** 31 - 1, 0),
                                  (fa.FA_MASK_CAUSAL_WINDOW, 2 ** 31 - 1, 2 ** 31 - 1),
                                  (fa.FA_MASK_BAND, 2 ** 31 - 1, 0),
                                  (fa.FA_MASK_PREFIX_LM, 0, 2 ** 31 - 1)], ids=str)
@pytest.mark.parametrize("lens_q,lens_k", [([200, 3], [3, 200]), ([5], [2])], ids=str)
def test_the_largest_windows_with_more_queries_than_keys(lens_q, lens_k, mask):
    """Queries before the first key make positions negative: a window takes them out of 32 bits."""
    H, Hkv, d = 4, 2, 64
    q, k, v, cu_q, cu_k = case(lens_q, lens_k, H, Hkv, d, torch.float16, seed=7)
    ref = attention(q, k, v, cu_q, cu_k, 0.125, *mask)
    o, lse = forward(q.cuda(), k.cuda(), v.cuda(), cu_q, cu_k, 0.125, mask)
    check_forward(o, lse, ref, torch.float16, sum(lens_q))
    page = 16  # the same keys in a cache, for few rows and for many
    width = -(-max(lens_k) // page)
    kp = torch.zeros(len(lens_k) * width, Hkv, page, d, dtype=torch.float16)
    vp = torch.zeros_like(kp)
    for b, n in enumerate(lens_k):
        for j in range(n):
            kp[b * width + j // page, :, j % page] = k[cu_k[b] + j]
            vp[b * width + j // page, :, j % page] = v[cu_k[b] + j]
    table = torch.arange(len(lens_k) * width, dtype=torch.int32).reshape(-1, width)
    o, lse = run_paged(q, kp, vp, table, lens_k, cu_q, max(lens_q), 0.125, mask)
    assert fa.fa_get_device_status() == fa.FA_OK
    check_forward(o, lse, ref, torch.float16, sum(lens_q))


@pytest.mark.parametrize("G", [1, 2, 3, 8, 12, 33, 64, 100, 128])
def test_group_sizes(G):
    lens = [70, 3, 150]
    q, k, v, cu, _ = case(lens, lens, G, 1, 64, torch.float16, seed=G)
    o, lse = forward(q.cuda(), k.cuda(), v.cuda(), cu, cu, 0.125)
    check_forward(o, lse, attention(q, k, v, cu, cu, 0.125, fa.FA_MASK_CAUSAL), torch.float16,
                  sum(lens), f"G={G}")


def test_slices_of_a_fused_projection_and_wider_outputs():
    H, Hkv, d, lens = 6, 2, 64, [40, 129]
    g = torch.Generator().manual_seed(1)
    qkv = torch.randn(sum(lens), H + 2 * Hkv, d, generator=g).to(torch.bfloat16)
    x = qkv.cuda()
    q, k, v = x[:, :H], x[:, H:H + Hkv], x[:, H + Hkv:]
    cu = starts(lens)
    wide = torch.full((sum(lens), H + 1, d), 5.0, dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(fa.fa_varlen_workspace_size(2, H, Hkv, sum(lens), sum(lens), d),
                     dtype=torch.uint8, device="cuda")
    fa.fa_fwd_varlen(q, k, v, wide[:, 1:], None, i32(cu), i32(cu), 0.125, ws)
    ref = attention(qkv[:, :H], qkv[:, H:H + Hkv], qkv[:, H + Hkv:], cu, cu, 0.125,
                    fa.FA_MASK_CAUSAL)
    check_forward(wide[:, 1:], None, ref, torch.bfloat16, sum(lens))
    assert (wide[:, 0] == 5.0).all()


def test_infinities_of_one_sequence_stay_there():
    """NaN and infinities in another sequence's q, k, v, and in rows of nobody."""
    lens, H, Hkv, d = [100, 30, 200], 4, 2, 64
    q, k, v, cu, _ = case(lens, lens, H, Hkv, d, torch.float16, seed=3, pad=40)
    ref = attention(q, k, v, cu, cu, 0.125, fa.FA_MASK_CAUSAL)
    for t in (q, k, v):
        t[100:130] = float("nan")
        t[110] = float("inf")
        t[330:] = float("nan")
    o, lse = forward(q.cuda(), k.cuda(), v.cuda(), cu, cu, 0.125)
    for rows in (slice(0, 100), slice(130, 330)):
        check_forward(o[rows], lse[rows], tuple(r[rows] for r in ref), torch.float16, 10 ** 9)


def test_same_bits_on_every_run():
    H, Hkv, d = 8, 2, 128
    q, k, v, cu, _ = case([500, 77], [500, 77], H, Hkv, d, torch.bfloat16, seed=4)
    qg, kg, vg = q.cuda(), k.cuda(), v.cuda()
    o1, l1 = forward(qg, kg, vg, cu, cu, 0.09)
    o2, l2 = forward(qg, kg, vg, cu, cu, 0.09)
    assert torch.equal(o1, o2) and torch.equal(l1, l2)


def test_captured_call_follows_new_lengths():
    H, Hkv, d, T = 4, 1, 64, 300
    q, k, v, _, _ = case([T], [T], H, Hkv, d, torch.float16, seed=5)
    qg, kg, vg = q.cuda(), k.cuda(), v.cuda()
    cu = i32([0, 100, 300])
    o = torch.zeros(T, H, d, dtype=torch.float16, device="cuda")
    lse = torch.zeros(T, H, device="cuda")
    ws = torch.empty(fa.fa_varlen_workspace_size(2, H, Hkv, T, T, d), dtype=torch.uint8,
                     device="cuda")
    fa.fa_fwd_varlen(qg, kg, vg, o, lse, cu, cu, 0.125, ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        fa.fa_fwd_varlen(qg, kg, vg, o, lse, cu, cu, 0.125, ws)
    for split in (100, 1, 0, 299):
        cu.copy_(i32([0, split, 300]))
        o.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        c = [0, split, 300]
        check_forward(o, lse, attention(q, k, v, c, c, 0.125, fa.FA_MASK_CAUSAL), torch.float16,
                      T, f"split {split}")


def test_bad_starts_are_reported_and_read_nothing():
    H, Hkv, d, T = 2, 1, 64, 64
    q, k, v, _, _ = case([T], [T], H, Hkv, d, torch.float16, seed=6)
    qg, kg, vg = q.cuda(), k.cuda(), v.cuda()
    for cu in ([0, 40, 65], [0, 40, 20], [-1, 20, 64]):
        o = torch.full((T, H, d), float("nan"), dtype=torch.float16, device="cuda")
        ws = torch.empty(fa.fa_varlen_workspace_size(2, H, Hkv, T, T, d), dtype=torch.uint8,
                         device="cuda")
        fa.fa_fwd_varlen(qg, kg, vg, o, None, i32(cu), i32(cu), 0.125, ws)
        assert fa.fa_get_device_status() == fa.FA_ERR_BAD_PAGE
        good = [(a, b) for a, b in zip(cu, cu[1:]) if 0 <= a <= b <= T]
        for a, b in good:
            ref = attention(q, k, v, [a, b], [a, b], 0.125, fa.FA_MASK_CAUSAL)
            check_forward(o[a:b], None, tuple(r[a:b] for r in ref), torch.float16, 10 ** 9)
        rows = torch.ones(T, dtype=torch.bool)
        for a, b in good:
            rows[a:b] = False
        assert o[rows.cuda()].isnan().all()


# ------------------------------------------------------------------ over a paged cache

def paged_case(new, before, H, Hkv, d, page, dtype, seed, pad=2):
    """Chunks of new tokens over caches of before[b] + new[b] keys; unused slots are NaN."""
    g = torch.Generator().manual_seed(seed)
    total = [n + c for n, c in zip(new, before)]
    need = [-(-t // page) for t in total]
    width, pages = max(need + [1]) + 1, sum(need) + 4
    perm = torch.randperm(pages, generator=g).tolist()
    table = torch.full((len(new), width), -1, dtype=torch.int32)
    kp = torch.full((pages, Hkv, page, d), float("nan"), dtype=dtype)
    vp = kp.clone()
    q = torch.randn(sum(new) + pad, H, d, generator=g).to(dtype)
    k = torch.randn(sum(total), Hkv, d, generator=g).to(dtype)
    v = torch.randn(sum(total), Hkv, d, generator=g).to(dtype)
    cu_k, at = starts(total), 0
    for b, n in enumerate(need):
        table[b, :n] = torch.tensor(perm[at:at + n], dtype=torch.int32)
        at += n
        pos = torch.arange(total[b])
        phys, slot = table[b, pos // page].long(), pos % page
        kp[phys, :, slot] = k[cu_k[b]:cu_k[b + 1]]
        vp[phys, :, slot] = v[cu_k[b]:cu_k[b + 1]]
    return q, k, v, kp, vp, table, total, starts(new), cu_k


def run_paged(q, kp, vp, table, total, cu, max_q, scale, mask=(fa.FA_MASK_CAUSAL, 0, 0)):
    T, H, d = q.shape
    o = torch.full((T, H, d), float("nan"), dtype=q.dtype, device="cuda")
    lse = torch.full((T, H), float("nan"), device="cuda")
    B, width = table.shape
    ws = torch.empty(fa.fa_paged_varlen_workspace_size(B, H, kp.shape[1], T, max_q, width,
                                                       kp.shape[2], d),
                     dtype=torch.uint8, device="cuda")
    fa.fa_fwd_paged_varlen(q.cuda(), kp.cuda(), vp.cuda(), table.cuda(), i32(total), i32(cu),
                           max_q, o, lse, scale, ws, *mask)
    return o, lse


PAGED = [([1, 1, 1], [0, 17, 300]), ([1], [4000]), ([3, 1, 0, 4], [60, 0, 9, 127]),
         ([16, 2, 9], [1000, 1, 0]), ([130, 1, 64], [70, 2000, 0]), ([300], [5])]


@pytest.mark.parametrize("new,before", PAGED, ids=str)
@pytest.mark.parametrize("H,Hkv,d,page,dt", [(4, 4, 64, 16, "f16"), (8, 2, 128, 256, "bf16"),
                                             (7, 1, 128, 64, "f16"), (10, 2, 64, 48, "bf16"),
                                             (16, 1, 128, 128, "bf16")])
@pytest.mark.parametrize("mask", ["none", "causal", "window"])
def test_paged_chunks(new, before, H, Hkv, d, page, dt, mask):
    q, k, v, kp, vp, table, total, cu, cu_k = paged_case(new, before, H, Hkv, d, page, DT[dt],
                                                         seed=sum(new) + page)
    scale = 1 / math.sqrt(d)
    o, lse = run_paged(q, kp, vp, table, total, cu, max(new), scale, MASKS[mask])
    assert fa.fa_get_device_status() == fa.FA_OK
    T = sum(new)
    check_forward(o, lse, attention(q, k, v, cu, cu_k, scale, *MASKS[mask]), DT[dt], T,
                  f"{new} {before} {mask}")
    assert o[T:].isnan().all() and lse[T:].isnan().all()


@pytest.mark.parametrize("new", [1, 40])
def test_paged_lengths_and_pages_out_of_range(new):
    """A length beyond the table is cut to it, a page outside the pool is read as page 0, and
    both are reported; a chunk longer than the keys leaves its first rows empty."""
    H, Hkv, d, page = 4, 2, 64, 16
    q, k, v, kp, vp, table, total, cu, cu_k = paged_case([new], [60], H, Hkv, d, page,
                                                         torch.float16, seed=1)
    kp, vp = kp.nan_to_num(0.5), vp.nan_to_num(0.5)
    full = table.clone()
    full[full < 0] = 0
    o, _ = run_paged(q, kp, vp, full, [10 ** 6], cu, new, 0.125)
    assert fa.fa_get_device_status() == fa.FA_ERR_BAD_PAGE
    want, _ = run_paged(q, kp, vp, full, [full.shape[1] * page], cu, new, 0.125)
    assert fa.fa_get_device_status() == fa.FA_OK
    assert torch.equal(o[:new], want[:new])
    bad, zero = table.clone(), table.clone()
    bad[0, 1], zero[0, 1] = kp.shape[0], 0
    o, _ = run_paged(q, kp, vp, bad, total, cu, new, 0.125)
    assert fa.fa_get_device_status() == fa.FA_ERR_BAD_PAGE
    want, _ = run_paged(q, kp, vp, zero, total, cu, new, 0.125)
    assert torch.equal(o[:new], want[:new])
    few = max(0, new - 5)  # queries sit at the last positions: the first 5 before the first key
    o, lse = run_paged(q, kp, vp, full, [few], cu, new, 0.125)
    assert fa.fa_get_device_status() == fa.FA_OK
    assert (o[:new - few] == 0).all() and lse[:new - few].isneginf().all()
    assert torch.isfinite(lse[new - few:new]).all()


@pytest.mark.parametrize("new", [1, 40])
def test_pages_beyond_32_bit_offsets(new):
    """A pool of 2.3e9 elements whose last pages hold the sequence."""
    H, Hkv, d, page, dt = 4, 2, 128, 64, torch.float16
    pages = 140000
    q, k, v, kp, vp, table, total, cu, cu_k = paged_case([new], [300], H, Hkv, d, page, dt, seed=2)
    shift = pages - kp.shape[0]
    assert pages * Hkv * page * d > 2 ** 31
    big_k, big_v = (torch.empty(pages, Hkv, page, d, dtype=dt, device="cuda") for _ in range(2))
    big_k[shift:], big_v[shift:] = kp.cuda(), vp.cuda()
    far = torch.where(table >= 0, table + shift, table)
    o = torch.full((new + 2, H, d), float("nan"), dtype=dt, device="cuda")
    lse = torch.full((new + 2, H), float("nan"), device="cuda")
    ws = torch.empty(fa.fa_paged_varlen_workspace_size(1, H, Hkv, new + 2, new, far.shape[1], page,
                                                       d), dtype=torch.uint8, device="cuda")
    fa.fa_fwd_paged_varlen(q.cuda(), big_k, big_v, far.cuda(), i32(total), i32(cu), new, o, lse,
                           0.09, ws)
    assert fa.fa_get_device_status() == fa.FA_OK
    check_forward(o, lse, attention(q, k, v, cu, cu_k, 0.09, fa.FA_MASK_CAUSAL), dt, new)


def test_two_streams_at_once():
    """Calls of two shapes that overlap, each on its own stream with its own workspace."""
    cases = []
    for i, (lens, H, Hkv, d) in enumerate([([700, 33], 8, 2, 128), ([64] * 9, 6, 3, 64)]):
        q, k, v, cu, _ = case(lens, lens, H, Hkv, d, torch.bfloat16, seed=i)
        args = [x.cuda() for x in (q, k, v)]
        want = forward(*args, cu, cu, 0.1)
        T = sum(lens)
        o = torch.zeros(T, H, d, dtype=torch.bfloat16, device="cuda")
        lse = torch.zeros(T, H, device="cuda")
        ws = torch.empty(fa.fa_varlen_workspace_size(len(lens), H, Hkv, T, T, d),
                         dtype=torch.uint8, device="cuda")
        cases.append((args, i32(cu), o, lse, ws, want, torch.cuda.Stream()))
    torch.cuda.synchronize()
    for _ in range(20):
        for args, cu, o, lse, ws, _, stream in cases:
            fa.fa_fwd_varlen(*args, o, lse, cu, cu, 0.1, ws, stream=stream)
    torch.cuda.synchronize()
    assert fa.fa_get_device_status() == fa.FA_OK
    for _, _, o, lse, _, want, _ in cases:
        assert torch.equal(o, want[0]) and torch.equal(lse, want[1])


def test_many_calls_in_a_row_without_waiting():
    """A few hundred calls queued at once over three sets of buffers, few rows and many."""
    H, Hkv, d, page, dt = 8, 2, 128, 64, torch.bfloat16
    for new, before in (([1] * 6, [0, 100, 3000, 64, 63, 700]), ([90, 3, 200], [800, 2000, 0])):
        sets = []
        for i in range(3):
            q, k, v, kp, vp, table, total, cu, _ = paged_case(new, before, H, Hkv, d, page, dt,
                                                              seed=i)
            want = run_paged(q, kp, vp, table, total, cu, max(new), 0.09)
            T = q.shape[0]
            ws = torch.empty(fa.fa_paged_varlen_workspace_size(len(new), H, Hkv, T, max(new),
                                                               table.shape[1], page, d),
                             dtype=torch.uint8, device="cuda")
            sets.append((q.cuda(), kp.cuda(), vp.cuda(), table.cuda(), i32(total), i32(cu),
                         torch.zeros_like(want[0]), torch.zeros_like(want[1]), ws, want))
        for i in range(300):
            q, kp, vp, table, ctx, cu, o, lse, ws, _ = sets[i % 3]
            fa.fa_fwd_paged_varlen(q, kp, vp, table, ctx, cu, max(new), o, lse, 0.09, ws)
        assert fa.fa_get_device_status() == fa.FA_OK
        n = sum(new)
        for *_, o, lse, _, want in sets:
            assert torch.equal(o[:n], want[0][:n]) and torch.equal(lse[:n], want[1][:n])


def test_long_sequence_of_many_units():
    """More token blocks than the plan kernel has threads, and more sequences too."""
    lens = [1] * 1500 + [0] * 7 + [3] * 40
    q, k, v, cu, _ = case(lens, lens, 2, 1, 64, torch.float16, seed=8)
    o, lse = forward(q.cuda(), k.cuda(), v.cuda(), cu, cu, 0.125)
    check_forward(o, lse, attention(q, k, v, cu, cu, 0.125, fa.FA_MASK_CAUSAL), torch.float16,
                  sum(lens))
    T = 40000  # 64 tokens a unit at 4 heads a group ... 32 at 8
    g = torch.Generator().manual_seed(1)
    q = torch.randn(T, 8, 64, generator=g).to(torch.float16)
    k, v = (torch.randn(T, 1, 64, generator=g).to(torch.float16) for _ in range(2))
    o, lse = forward(q.cuda(), k.cuda(), v.cuda(), [0, T], [0, T], 0.125,
                     (fa.FA_MASK_CAUSAL_WINDOW, 100, 3))
    for a in (0, 20001, T - 300):  # windows of queries with the keys that they can see
        lo = max(0, a - 100)
        keys = list(range(3)) + list(range(max(3, lo), a + 300)) if lo > 3 else range(a + 300)
        i, j = torch.arange(a, a + 300)[:, None], torch.tensor(list(keys))[None]
        vis = (j <= i) & ((i - j < 100) | (j < 3))
        from _packed import head
        _, want, wl = head(q[a:a + 300, 5], k[j[0], 0], v[j[0], 0], vis, 0.125)
        big = (vis * v[j[0], 0].double().abs().amax(-1)[None]).amax(-1)
        ref = (want[:, None], wl[:, None], big[:, None])
        check_forward(o[a:a + 300, 5:6], lse[a:a + 300, 5:6], ref, torch.float16, 300, f"from {a}")


def test_python_refusals():
    H, Hkv, d, T = 4, 2, 64, 10
    q, k, v, cu, _ = case([T], [T], H, Hkv, d, torch.float16, seed=1)
    q, k, v, cu = q.cuda(), k.cuda(), v.cuda(), i32(cu)
    o = torch.empty_like(q)
    ws = torch.empty(fa.fa_varlen_workspace_size(1, H, Hkv, T, T, d), dtype=torch.uint8,
                     device="cuda")
    good = dict(q=q, k=k, v=v, o=o, lse=None, cu_seqlens_q=cu, cu_seqlens_k=cu, scale=0.125,
                workspace=ws)
    fa.fa_fwd_varlen(**good)
    bad = [dict(cu_seqlens_q=cu.long()), dict(k=k.bfloat16()), dict(v=v[:-1]), dict(o=o[:, :2]),
           dict(q=q.transpose(0, 1)), dict(k=k[:, :1].expand(T, Hkv, d)), dict(q=q.cpu()),
           dict(workspace=ws[:16]), dict(lse=torch.empty(T, H + 1, device="cuda")),
           dict(cu_seqlens_k=cu[:1]), dict(lse=torch.empty(T, H, device="cuda").half())]
    for kw in bad:
        with pytest.raises(fa.FaError):
            fa.fa_fwd_varlen(**dict(good, **kw))


@pytest.mark.parametrize("new", [1, 3, 5, 40, 100])
@pytest.mark.parametrize("dt", list(DT))
def test_scores_that_climb(new, dt):
    """Every later block lifts every row's maximum by more than the lazy-rescale threshold (12 in
    log2 units a block of 128 keys, as in inputs.climbing_inputs), for few rows, items of one tile
    and of two; and their falling mirror image."""
    H, Hkv, d, page, ctx = 8, 1, 64, 64, 1500
    for sign in (1.0, -1.0):
        q, k, v, kp, vp, table, total, cu, cu_k = paged_case([new], [ctx], H, Hkv, d, page, DT[dt],
                                                             seed=new)
        T = total[0]
        # q = N(0,1) + 1, k_j = N(0,1) + a_j: the mean score rises by scale d a_j = 8 a_j
        q = (q.float() + 1).to(DT[dt])
        a = sign * torch.arange(T).float() / 128 * (12 * math.log(2) / 8)
        k = (k.float() + a[:, None, None]).to(DT[dt])
        pos = torch.arange(T)
        kp[table[0, pos // page].long(), :, pos % page] = k
        o, lse = run_paged(q, kp, vp, table, total, cu, new, 0.125)
        assert fa.fa_get_device_status() == fa.FA_OK
        ref = attention(q, k, v, cu, cu_k, 0.125, fa.FA_MASK_CAUSAL)
        # |scores| reach 130 here: the FP32 products' and sums' error grows with them (2^-24 of a
        # sum of |q k| up to 300 in 64 terms: 2^-13), and the weights' by as much
        check_forward(o, None, (ref[0], ref[1], ref[2] * (1 + 2.0 ** -4)), DT[dt], new)
        assert float((lse[:new].double().cpu() - ref[1][:new]).abs().max()) <= 2.0 ** -10


@pytest.mark.parametrize("H,Hkv", [(4, 2), (32, 1)])
def test_more_sequences_than_the_plan_has_threads(H, Hkv):
    """1500 sequences of 0 to 3 tokens: by themselves and as chunks over a cache."""
    d, dt = 64, torch.float16
    lens = [(5 * b) % 4 for b in range(1500)]
    q, k, v, cu, _ = case(lens, lens, H, Hkv, d, dt, seed=9, pad=1)
    o, lse = forward(q.cuda(), k.cuda(), v.cuda(), cu, cu, 0.125)
    check_forward(o, lse, attention(q, k, v, cu, cu, 0.125, fa.FA_MASK_CAUSAL), dt, sum(lens))
    assert o[sum(lens):].isnan().all()
    before = [(7 * b) % 40 for b in range(1500)]
    q, k, v, kp, vp, table, total, cu, cu_k = paged_case(lens, before, H, Hkv, d, 16, dt, seed=9)
    o, lse = run_paged(q, kp, vp, table, total, cu, 3, 0.125)
    assert fa.fa_get_device_status() == fa.FA_OK
    check_forward(o, lse, attention(q, k, v, cu, cu_k, 0.125, fa.FA_MASK_CAUSAL), dt, sum(lens))
    assert o[sum(lens):].isnan().all() and lse[sum(lens):].isnan().all()


@pytest.mark.parametrize("max_q", [3, 40])
def test_captured_paged_call_follows_lengths_pages_and_chunks(max_q):
    """One graph, replayed after the lengths, the table and the chunks have changed."""
    H, Hkv, d, page, dt = 8, 2, 128, 16, torch.bfloat16
    B, width, T = 3, 30, 3 * max_q
    o = torch.zeros(T, H, d, dtype=dt, device="cuda")
    lse = torch.zeros(T, H, device="cuda")
    pool = torch.zeros(B * width + 4, Hkv, page, d, dtype=dt, device="cuda")
    kp, vp, q = pool, pool.clone(), torch.zeros_like(o)
    table = torch.zeros(B, width, dtype=torch.int32, device="cuda")
    ctx, cu = i32([0] * B), i32([0] * (B + 1))
    ws = torch.empty(fa.fa_paged_varlen_workspace_size(B, H, Hkv, T, max_q, width, page, d),
                     dtype=torch.uint8, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        fa.fa_fwd_paged_varlen(q, kp, vp, table, ctx, cu, max_q, o, lse, 0.09, ws)
    for new, before in (([1, 1, 1], [9, 0, 400]), ([3, 0, 2], [60, 17, 1]),
                        ([max_q, 1, max_q], [200, 3, 5]), ([0, 0, 0], [4, 5, 6])):
        qc, kc, vc, kpc, vpc, tc, total, cuc, cu_k = paged_case(new, before, H, Hkv, d, page, dt,
                                                                seed=sum(before), pad=0)
        q[:sum(new)] = qc.cuda()
        kp[:kpc.shape[0]], vp[:vpc.shape[0]] = kpc.cuda(), vpc.cuda()
        table.fill_(-1)
        table[:, :tc.shape[1]] = tc.cuda()
        ctx.copy_(i32(total))
        cu.copy_(i32(cuc))
        o.fill_(float("nan"))
        lse.fill_(float("nan"))
        graph.replay()
        assert fa.fa_get_device_status() == fa.FA_OK
        check_forward(o, lse, attention(qc, kc, vc, cuc, cu_k, 0.09, fa.FA_MASK_CAUSAL), dt,
                      sum(new), f"{new} {before}")
        assert o[sum(new):].isnan().all() and lse[sum(new):].isnan().all()


@pytest.mark.parametrize("new", [2, 50])
def test_masks_that_leave_rows_of_a_cached_chunk_empty(new):
    """A band over fewer keys than queries: rows far before the first key see nothing."""
    H, Hkv, d, page, dt = 4, 2, 64, 16, torch.float16
    keys = max(1, new // 5)
    q, k, v, cu_q, cu_k = case([new, new], [keys, keys], H, Hkv, d, dt, seed=new)
    kp = torch.full((2, Hkv, page, d), float("nan"), dtype=dt)
    vp = kp.clone()
    for b in range(2):
        kp[b, :, :keys] = k[b * keys:(b + 1) * keys].transpose(0, 1)
        vp[b, :, :keys] = v[b * keys:(b + 1) * keys].transpose(0, 1)
    table = torch.tensor([[0], [1]], dtype=torch.int32)
    mask = (fa.FA_MASK_BAND, 0, 0)
    o, lse = run_paged(q, kp, vp, table, [keys, keys], cu_q, new, 0.125, mask)
    assert fa.fa_get_device_status() == fa.FA_OK
    check_forward(o, lse, attention(q, k, v, cu_q, cu_k, 0.125, *mask), dt, 2 * new)


def test_python_refusals_of_shapes_and_numbers():
    """Wrong dimensions and numbers that a field does not hold raise FaError in every call."""
    H, Hkv, d, T, page = 4, 2, 64, 10, 16
    q, k, v, cu, _ = case([T], [T], H, Hkv, d, torch.float16, seed=1)
    q, k, v, cu = q.cuda(), k.cuda(), v.cuda(), i32(cu)
    o, lse = torch.empty_like(q), torch.empty(T, H, device="cuda")
    kp = torch.zeros(2, Hkv, page, d, dtype=torch.float16, device="cuda")
    table, ctx = i32([[0, 1]]), i32([0])
    freqs, _ = fa.fa_rope_freqs(d, device="cuda")
    ws = torch.empty(max(fa.fa_varlen_workspace_size(1, H, Hkv, T, T, d),
                         fa.fa_bwd_varlen_workspace_size(1, H, Hkv, T, T, d),
                         fa.fa_paged_varlen_workspace_size(1, H, Hkv, T, T, 2, page, d)),
                     dtype=torch.uint8, device="cuda")
    mask = [dict(window=2 ** 40), dict(n_global=2 ** 31), dict(mask_mode=-2 ** 31 - 1),
            dict(scale=1e300), dict(q=q[0]), dict(q=q[None]), dict(o=o[:, 0]), dict(o=o[:-1]),
            dict(lse=lse[0])]
    kv = [dict(k=k[0]), dict(k=k[None]), dict(v=v[:, 0]), dict(v=v[:-1]),
          dict(cu_seqlens_k=cu[:1]), dict(cu_seqlens_k=cu[None]), dict(cu_seqlens_q=cu[0])]
    pools = [dict(k_pages=kp[0]), dict(v_pages=kp[0]), dict(k_pages=kp[None]),
             dict(block_table=table[0]), dict(ctx_lens=ctx[None])]
    packed = dict(q=q, k=k, v=v, o=o, lse=lse, cu_seqlens_q=cu, cu_seqlens_k=cu, scale=0.125,
                  workspace=ws)
    grads = dict(dout=torch.zeros_like(q), dq=torch.empty_like(q), dk=torch.empty_like(k),
                 dv=torch.empty_like(v))
    x = torch.empty(T, H, d, dtype=torch.float16, device="cuda")
    for call, good, bad in (
            (fa.fa_fwd_varlen, packed, mask + kv),
            (fa.fa_bwd_varlen, dict(packed, **grads), mask + kv + [
                {n: t[0]} for n, t in grads.items()] + [{n: t[:-1]} for n, t in grads.items()]),
            (fa.fa_fwd_paged_varlen,
             dict(q=q, k_pages=kp, v_pages=kp, block_table=table, ctx_lens=i32([T]),
                  cu_seqlens_q=cu, max_q=T, o=o, lse=lse, scale=0.125, workspace=ws),
             mask + pools + [dict(max_q=2 ** 31), dict(max_q=2.0), dict(cu_seqlens_q=cu[0])]),
            (fa.fa_rope_append,
             dict(q=q, k=k, v=v, q_out=x, k_pages=kp, v_pages=kp.clone(), block_table=table,
                  ctx_lens=ctx, cu_seqlens=cu, freqs=freqs),
             pools + [dict(q=q[0]), dict(k=k[:-1]), dict(v=v[0]), dict(q_out=x[:-1]),
                      dict(style=2 ** 32), dict(amplitude=1e300), dict(freqs=freqs[0]),
                      dict(cu_seqlens=cu[0])]),
            (fa.fa_rope, dict(x=q, y=x, positions=i32(list(range(T))), freqs=freqs),
             [dict(style=2 ** 32), dict(x=q[0]), dict(y=x[0]), dict(positions=cu),
              dict(freqs=freqs[0]), dict(freqs=freqs[None]), dict(amplitude=1e300)])):
        call(**good)
        for kw in bad:
            with pytest.raises(fa.FaError):
                call(**dict(good, **kw))
    assert fa.fa_get_device_status() == fa.FA_OK


def check_nan_rows(o, lse, hit, T):
    """Rows (token, head) of `hit` are NaN in o and lse, every other of the T tokens is finite."""
    want = torch.zeros(T, o.shape[1], dtype=torch.bool)
    for t, h in hit:
        want[t, h] = True
    assert torch.equal(o[:T].isnan().all(-1).cpu(), want)
    assert torch.equal(o[:T].isfinite().all(-1).cpu(), ~want)
    assert torch.equal(lse[:T].isnan().cpu(), want)
    assert torch.equal(lse[:T].isfinite().cpu(), ~want)


@pytest.mark.parametrize("lens", [[300, 40, 3], [4000]], ids=str)
@pytest.mark.parametrize("d,dt", [(64, "f16"), (128, "bf16")])
def test_a_row_of_nan_scores_has_a_nan_lse(lens, d, dt):
    """An -inf there would say that the row sees no key. Whole tiles, partial ones, split items."""
    H, Hkv, T = 4, 2, sum(lens)
    q, k, v, cu, _ = case(lens, lens, H, Hkv, d, DT[dt], seed=1)
    hit = [(0, 1), (257, 3), (T - 1, 0)]
    for t, h in hit:
        q[t, h, t % d] = float("nan")
    o, lse = forward(q.cuda(), k.cuda(), v.cuda(), cu, cu, 1 / math.sqrt(d))
    check_nan_rows(o, lse, hit, T)


@pytest.mark.parametrize("new,before", [([1, 2], [300, 5000]), ([40, 3], [30, 5000])], ids=str)
def test_a_row_of_nan_scores_over_a_cache_has_a_nan_lse(new, before):
    """Few rows (whole pairs and joined pieces) and the 128-row tiles."""
    q, _, _, kp, vp, table, total, cu, _ = paged_case(new, before, 4, 2, 64, 16, torch.float16, 3)
    T = sum(new)
    hit = [(0, 1), (T - 1, 2)]
    for t, h in hit:
        q[t, h, 5] = float("nan")
    o, lse = run_paged(q, kp, vp, table, total, cu, max(new), 0.125)
    assert fa.fa_get_device_status() == fa.FA_OK
    check_nan_rows(o, lse, hit, T)


@pytest.mark.parametrize("cu", [[0, 5, 13], [0, 6, 4], [-1, 6, 12], [0, 3, 6, -5, 12],
                                [0, 3, 6, 2 ** 31 - 1, 12], [6, 12, 0, 6]], ids=str)
@pytest.mark.parametrize("max_q", [6, 60])
def test_bad_starts_over_a_cache_are_reported_and_leave_others(cu, max_q):
    """For few rows and for the 128-row tiles."""
    H, Hkv, d, page, T, B = 4, 2, 64, 16, 12, len(cu) - 1
    good = [0 <= a <= b <= T for a, b in zip(cu, cu[1:])]
    new = [b - a if ok else 0 for a, b, ok in zip(cu, cu[1:], good)]
    q, k, v, kp, vp, table, total, _, cu_k = paged_case(new, [40 + 70 * b for b in range(B)], H, Hkv,
                                                       d, page, torch.float16, seed=2)
    q = torch.randn(T, H, d, generator=torch.Generator().manual_seed(3)).half()
    o, lse = run_paged(q, kp, vp, table, total, cu, max_q, 0.125)
    assert fa.fa_get_device_status() == fa.FA_ERR_BAD_PAGE
    rows = torch.ones(T, dtype=torch.bool)
    for b in range(B):
        if good[b]:
            a, e, keys = cu[b], cu[b + 1], slice(cu_k[b], cu_k[b + 1])
            rows[a:e] = False
            ref = attention(q[a:e], k[keys], v[keys], [0, e - a], [0, total[b]], 0.125,
                            fa.FA_MASK_CAUSAL)
            check_forward(o[a:e], lse[a:e], ref, torch.float16, e - a, f"{cu} {b}")
    assert o[rows.cuda()].isnan().all() and lse[rows.cuda()].isnan().all()
