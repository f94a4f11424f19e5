"""Gradients of packed grouped-head attention through the C ABI: against the formula in 64 bits
with bounds that count the roundings (_packed.py), against differences, and the run of rotation,
attention, their gradients and the paged cache as a training and a serving step use them."""
import math

import pytest
import torch

import tiled_attention_06_gb300 as fa

from _packed import attention, check_forward, check_gradients, gradients, rotate, starts

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


def step(q, k, v, dout, cu_q, cu_k, scale, mask=(fa.FA_MASK_CAUSAL, 0, 0)):
    """Forward and backward of GPU tensors; outputs poisoned first."""
    T, H, d = q.shape
    Tk, Hkv, _ = k.shape
    B = len(cu_q) - 1
    o = torch.full((T, H, d), float("nan"), dtype=q.dtype, device="cuda")
    lse = torch.full((T, H), float("nan"), device="cuda")
    dq = torch.full((T, H, d), float("nan"), dtype=q.dtype, device="cuda")
    dk, dv = (torch.full((Tk, Hkv, d), float("nan"), dtype=q.dtype, device="cuda")
              for _ in range(2))
    size = max(fa.fa_varlen_workspace_size(B, H, Hkv, T, Tk, d),
               fa.fa_bwd_varlen_workspace_size(B, H, Hkv, T, Tk, d), 16)
    ws = torch.full((size,), 255, dtype=torch.uint8, device="cuda")  # NaNs: contents do not matter
    cq, ck = i32(cu_q), i32(cu_k)
    fa.fa_fwd_varlen(q, k, v, o, lse, cq, ck, scale, ws, *mask)
    ws.fill_(255)
    fa.fa_bwd_varlen(q, k, v, o, dout, lse, dq, dk, dv, cq, ck, scale, ws, *mask)
    assert fa.fa_get_device_status() == fa.FA_OK
    return dq, dk, dv


def case(lens_q, lens_k, H, Hkv, d, dtype, seed, pad=0):
    g = torch.Generator().manual_seed(seed)
    q, dout = (torch.randn(sum(lens_q) + pad, H, d, generator=g).to(dtype) for _ in range(2))
    k, v = (torch.randn(sum(lens_k) + pad, Hkv, d, generator=g).to(dtype) for _ in range(2))
    return q, k, v, dout, starts(lens_q), starts(lens_k)


LENS = [[1], [1, 1, 1], [0, 5, 0], [128], [129, 1, 63], [17, 300, 64, 2]]


@pytest.mark.parametrize("lens", LENS, ids=str)
@pytest.mark.parametrize("H,Hkv,d,dt", [(4, 4, 64, "f16"), (8, 2, 128, "bf16"),
                                        (7, 1, 128, "f16"), (6, 2, 64, "bf16")])
@pytest.mark.parametrize("mask", list(MASKS))
def test_gradients_of_self_attention(lens, H, Hkv, d, dt, mask):
    q, k, v, dout, cu, _ = case(lens, lens, H, Hkv, d, DT[dt], seed=sum(lens) + H, pad=2)
    scale = 1 / math.sqrt(d)
    got = step(q.cuda(), k.cuda(), v.cuda(), dout.cuda(), cu, cu, scale, MASKS[mask])
    T = sum(lens)
    ref = gradients(q, k, v, dout, cu, cu, scale, DT[dt], *MASKS[mask])
    check_gradients(got, ref, T, T, f"{lens} {mask}")
    assert all(x[T:].isnan().all() for x in got)  # rows behind the last sequence


@pytest.mark.parametrize("lens_q,lens_k", [([3, 200, 1], [200, 3, 0]), ([1, 1], [1000, 129]),
                                           ([130, 0, 2], [0, 7, 260]), ([0], [70]),
                                           ([70], [0])], ids=str)
@pytest.mark.parametrize("G", [1, 5])
@pytest.mark.parametrize("mask", list(MASKS))
def test_gradients_with_other_keys_than_queries(lens_q, lens_k, G, mask):
    q, k, v, dout, cu_q, cu_k = case(lens_q, lens_k, 2 * G, 2, 128, torch.bfloat16, seed=G)
    got = step(q.cuda(), k.cuda(), v.cuda(), dout.cuda(), cu_q, cu_k, 0.09, MASKS[mask])
    ref = gradients(q, k, v, dout, cu_q, cu_k, 0.09, torch.bfloat16, *MASKS[mask])
    check_gradients(got, ref, sum(lens_q), sum(lens_k), f"{lens_q} {lens_k} {mask}")


@pytest.mark.parametrize("mask", [(fa.FA_MASK_CAUSAL_WINDOW, 2 ** 31 - 1, 0),
                                  (fa.FA_MASK_BAND, 2 ** 31 - 1, 0)], ids=str)
def test_gradients_of_the_largest_windows(mask):
    q, k, v, dout, cu_q, cu_k = case([200, 3], [3, 200], 4, 2, 64, torch.float16, seed=8)
    got = step(q.cuda(), k.cuda(), v.cuda(), dout.cuda(), cu_q, cu_k, 0.125, mask)
    ref = gradients(q, k, v, dout, cu_q, cu_k, 0.125, torch.float16, *mask)
    check_gradients(got, ref, 203, 203)


@pytest.mark.parametrize("G", [2, 3, 8, 12, 33, 64, 100, 128])
def test_gradients_for_group_sizes(G):
    lens = [70, 3, 150]
    q, k, v, dout, cu, _ = case(lens, lens, G, 1, 64, torch.float16, seed=G)
    got = step(q.cuda(), k.cuda(), v.cuda(), dout.cuda(), cu, cu, 0.125)
    ref = gradients(q, k, v, dout, cu, cu, 0.125, torch.float16, fa.FA_MASK_CAUSAL)
    check_gradients(got, ref, sum(lens), sum(lens), f"G={G}")


@pytest.mark.parametrize("lens", [[2000, 1300, 700], [5000]], ids=str)
def test_gradients_without_head_subsets_and_of_long_sequences(lens):
    """Enough key blocks for one head subset (16 K/V heads), and more halves than stages."""
    q, k, v, dout, cu, _ = case(lens, lens, 32, 16, 64, torch.bfloat16, seed=1)
    got = step(q.cuda(), k.cuda(), v.cuda(), dout.cuda(), cu, cu, 0.125)
    # one K/V head's worth of the reference is enough work for the CPU
    ref = gradients(q[:, 6:8], k[:, 3:4], v[:, 3:4], dout[:, 6:8], cu, cu, 0.125, torch.bfloat16,
                    fa.FA_MASK_CAUSAL)
    check_gradients((got[0][:, 6:8], got[1][:, 3:4], got[2][:, 3:4]), ref, sum(lens), sum(lens))


def test_infinities_of_one_sequence_stay_there():
    lens, H, Hkv, d = [100, 30, 200], 4, 2, 64
    q, k, v, dout, cu, _ = case(lens, lens, H, Hkv, d, torch.float16, seed=3, pad=40)
    ref = gradients(q, k, v, dout, cu, cu, 0.125, torch.float16, fa.FA_MASK_CAUSAL)
    for t in (q, k, v, dout):
        t[100:130] = float("nan")
        t[110] = float("inf")
        t[330:] = float("nan")
    got = step(q.cuda(), k.cuda(), v.cuda(), dout.cuda(), cu, cu, 0.125)
    for rows in (slice(0, 100), slice(130, 330)):
        check_gradients([x[rows] for x in got], [(r[rows], b[rows]) for r, b in ref], 10 ** 9,
                        10 ** 9)


@pytest.mark.parametrize("H,Hkv", [(4, 2), (32, 1)])
def test_gradients_of_more_sequences_than_the_plan_has_threads(H, Hkv):
    lens = [(5 * b) % 4 for b in range(1500)]
    q, k, v, dout, cu, _ = case(lens, lens, H, Hkv, 64, torch.float16, seed=9, pad=1)
    got = step(q.cuda(), k.cuda(), v.cuda(), dout.cuda(), cu, cu, 0.125)
    ref = gradients(q, k, v, dout, cu, cu, 0.125, torch.float16, fa.FA_MASK_CAUSAL)
    check_gradients(got, ref, sum(lens), sum(lens))
    assert all(x[sum(lens):].isnan().all() for x in got)


def test_slices_of_a_fused_projection_as_inputs_and_outputs():
    H, Hkv, d, lens = 6, 2, 64, [40, 129]
    T, cu = sum(lens), starts(lens)
    g = torch.Generator().manual_seed(1)
    qkv = torch.randn(T, H + 2 * Hkv, d, generator=g).to(torch.bfloat16)
    dout = torch.randn(T, H, d, generator=g).to(torch.bfloat16)
    x, dx = qkv.cuda(), torch.zeros_like(qkv, device="cuda")
    cut = lambda t: (t[:, :H], t[:, H:H + Hkv], t[:, H + Hkv:])  # noqa: E731
    o, lse = torch.empty(T, H, d, dtype=torch.bfloat16, device="cuda"), torch.empty(T, H).cuda()
    ws = torch.empty(max(fa.fa_varlen_workspace_size(2, H, Hkv, T, T, d),
                         fa.fa_bwd_varlen_workspace_size(2, H, Hkv, T, T, d)),
                     dtype=torch.uint8, device="cuda")
    fa.fa_fwd_varlen(*cut(x), o, lse, i32(cu), i32(cu), 0.125, ws)
    fa.fa_bwd_varlen(*cut(x), o, dout.cuda(), lse, *cut(dx), i32(cu), i32(cu), 0.125, ws)
    ref = gradients(*cut(qkv), dout, cu, cu, 0.125, torch.bfloat16, fa.FA_MASK_CAUSAL)
    check_gradients(cut(dx), ref, T, T)


def test_gradients_against_differences():
    """Central differences of the 64-bit forward along random directions: <grad, e> against
    (f(x + h e) - f(x - h e)) / 2h with h = 2^-10 (truncation h^2 times the third derivative,
    below 2^-14 here), the gradient's own error within its element bounds summed over e."""
    lens, H, Hkv, d, scale = [9, 4], 4, 2, 64, 0.125
    q, k, v, dout, cu, _ = case(lens, lens, H, Hkv, d, torch.float16, seed=9)
    got = step(q.cuda(), k.cuda(), v.cuda(), dout.cuda(), cu, cu, scale)
    bounds = gradients(q, k, v, dout, cu, cu, scale, torch.float16, fa.FA_MASK_CAUSAL)

    def loss(a, b, c):
        o, _, _ = attention(a, b, c, cu, cu, scale, fa.FA_MASK_CAUSAL)
        return float((o * dout.double()).sum())

    g, h = torch.Generator().manual_seed(2), 2.0 ** -10
    for i, x in enumerate((q, k, v)):
        e = torch.randint(0, 2, x.shape, generator=g).double() * 2 - 1
        args = [t.double() for t in (q, k, v)]
        up, down = list(args), list(args)
        up[i], down[i] = args[i] + h * e, args[i] - h * e
        diff = (loss(*up) - loss(*down)) / (2 * h)
        have = float((got[i].double().cpu() * e).sum())
        assert abs(have - diff) <= float(bounds[i][1].sum()) + 2.0 ** -14 * (1 + abs(diff))


def test_dk_and_dv_are_the_same_on_every_run():
    lens = [700, 33]
    q, k, v, dout, cu, _ = case(lens, lens, 8, 2, 128, torch.bfloat16, seed=4)
    args = [x.cuda() for x in (q, k, v, dout)]
    a, b = step(*args, cu, cu, 0.09), step(*args, cu, cu, 0.09)
    assert torch.equal(a[1], b[1]) and torch.equal(a[2], b[2])


def test_captured_backward_follows_new_lengths():
    H, Hkv, d, T = 4, 1, 64, 300
    q, k, v, dout, _, _ = case([T], [T], H, Hkv, d, torch.float16, seed=5)
    qg, kg, vg, dg = (x.cuda() for x in (q, k, v, dout))
    cu = i32([0, 100, 300])
    o = torch.zeros(T, H, d, dtype=torch.float16, device="cuda")
    lse = torch.zeros(T, H, device="cuda")
    dq, dk, dv = torch.zeros_like(qg), torch.zeros_like(kg), torch.zeros_like(vg)
    wf = torch.empty(fa.fa_varlen_workspace_size(2, H, Hkv, T, T, d), dtype=torch.uint8,
                     device="cuda")
    wb = torch.empty(fa.fa_bwd_varlen_workspace_size(2, H, Hkv, T, T, d), dtype=torch.uint8,
                     device="cuda")

    def both():
        fa.fa_fwd_varlen(qg, kg, vg, o, lse, cu, cu, 0.125, wf)
        fa.fa_bwd_varlen(qg, kg, vg, o, dg, lse, dq, dk, dv, cu, cu, 0.125, wb)
    both()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        both()
    for split in (100, 1, 0, 299):
        cu.copy_(i32([0, split, 300]))
        graph.replay()
        torch.cuda.synchronize()
        c = [0, split, 300]
        ref = gradients(q, k, v, dout, c, c, 0.125, torch.float16, fa.FA_MASK_CAUSAL)
        check_gradients((dq, dk, dv), ref, T, T, f"split {split}")


# ------------------------------------------------------------------ as they are used together

def test_training_step_of_rotated_attention():
    """Rotate q and k, attend, and go back: the gradient of the unrotated q and k is the inverse
    rotation of dq and dk. Each kernel is checked by itself above; here the chain is compared
    with the 64-bit chain, whose q and k are rounded after the rotation as the kernels' are."""
    H, Hkv, d, lens = 8, 2, 128, [200, 77]
    T, cu, scale, dt = sum(lens), starts(lens), 1 / math.sqrt(128), torch.bfloat16
    g = torch.Generator().manual_seed(1)
    qkv = torch.randn(T, H + 2 * Hkv, d, generator=g).to(dt)
    dout = torch.randn(T, H, d, generator=g).to(dt)
    pos = torch.cat([torch.arange(n) for n in lens]).to(torch.int32)
    freqs, amp = fa.fa_rope_freqs(d)
    fg, pg = freqs.cuda(), pos.cuda()
    x = qkv.cuda()
    qk = x[:, :H + Hkv]
    fa.fa_rope(qk, qk, pg, fg)  # in place, q and k at once
    q, k, v = x[:, :H], x[:, H:H + Hkv], x[:, H + Hkv:]
    dq, dk, dv = step(q, k, v, dout.cuda(), cu, cu, scale)
    fa.fa_rope(dq, dq, pg, fg, inverse=True)
    fa.fa_rope(dk, dk, pg, fg, inverse=True)
    rq, rk = q.cpu(), k.cpu()  # checked against the rotation in test_gpu_rope.py
    ref = gradients(rq, rk, qkv[:, H + Hkv:], dout, cu, cu, scale, dt, fa.FA_MASK_CAUSAL)
    u = torch.finfo(dt).eps / 2
    for got, (r, bound) in ((dq, ref[0]), (dk, ref[1])):
        want = rotate(r, pos, freqs, d, True, inverse=True)
        pair = bound + u * (r.abs() + bound)  # rounded again after the inverse rotation
        s = pair[..., :64] + pair[..., 64:] + 2 * u * (r[..., :64].abs() + r[..., 64:].abs())
        assert ((got.double().cpu() - want).abs() <= torch.cat([s, s], -1) + 2.0 ** -18).all()


def test_serving_chunks_then_single_tokens():
    """A prompt in ragged chunks, then single tokens, through fa_rope_append and
    fa_fwd_paged_varlen: every step's output against attention over the whole rotated prefix."""
    H, Hkv, d, page, dt = 8, 2, 64, 16, torch.bfloat16
    steps = [[33, 5], [20, 64], [1, 1], [1, 0], [1, 3]]
    B, width, scale = 2, 12, 0.125
    total = [sum(s[b] for s in steps) for b in range(B)]
    g = torch.Generator().manual_seed(3)
    table = torch.randperm(B * width + 3, generator=g)[:B * width].reshape(B, width)
    tg = table.to(torch.int32).cuda()
    kp = torch.full((B * width + 3, Hkv, page, d), float("nan"), dtype=dt, device="cuda")
    vp = kp.clone()
    freqs, amp = fa.fa_rope_freqs(d, scaling=fa.FA_ROPE_LINEAR, factor=2.0)
    fg = freqs.cuda()
    have, keys, vals = [0] * B, [[] for _ in range(B)], [[] for _ in range(B)]
    for new in steps:
        T, cu = sum(new), starts(new)
        qkv = torch.randn(T, H + 2 * Hkv, d, generator=g).to(dt)
        x = qkv.cuda()
        q_rot = torch.empty(T, H, d, dtype=dt, device="cuda")
        ctx = i32(have)
        fa.fa_rope_append(x[:, :H], x[:, H:H + Hkv], x[:, H + Hkv:], q_rot, kp, vp, tg, ctx,
                          i32(cu), fg)
        ctx += i32(new)
        o, lse = torch.empty_like(q_rot), torch.empty(T, H, device="cuda")
        ws = torch.empty(fa.fa_paged_varlen_workspace_size(B, H, Hkv, T, max(new), width, page, d),
                         dtype=torch.uint8, device="cuda")
        fa.fa_fwd_paged_varlen(q_rot, kp, vp, tg, ctx, i32(cu), max(new), o, lse, scale, ws)
        assert fa.fa_get_device_status() == fa.FA_OK
        for b in range(B):
            rows = slice(cu[b], cu[b + 1])
            pos = torch.arange(have[b], have[b] + new[b])
            at = (table[b, pos // page].long().cuda(), slice(None), (pos % page).cuda())
            keys[b].append(kp[at].cpu())  # the rotated keys as rounded into the cache
            want = rotate(qkv[rows, H:H + Hkv], pos, freqs, d, True)
            err = (keys[b][-1].double() - want).abs()
            mag = qkv[rows, H:H + Hkv].double().abs()
            s = mag[..., :32] + mag[..., 32:]
            assert (err <= torch.cat([s, s], -1) * (2.0 ** -8 + 2.0 ** -20) + 2.0 ** -24).all()
            vals[b].append(qkv[rows, H + Hkv:])
            have[b] += new[b]
        cu_k = starts(have)
        k, v = (torch.cat([torch.cat(s) for s in store]) for store in (keys, vals))
        check_forward(o, lse, attention(q_rot.cpu(), k, v, cu, cu_k, scale, fa.FA_MASK_CAUSAL), dt,
                      T, f"{new}")
    assert have == total


def bad_starts(B, seed):
    """Starts of B sequences of 0 to 7 tokens with bad ones: three below zero, one beyond the
    rows, and a decreasing one that is followed by another beyond the rows."""
    g = torch.Generator().manual_seed(seed)
    cu = starts(torch.randint(0, 8, (B,), generator=g).tolist())
    T = cu[-1]
    for b in (0, B // 3, B - 40):
        cu[b] = -7 - b
    cu[B // 2] = T + 50
    cu[B // 4], cu[B // 4 + 1] = 3, T + 9
    return cu, T


BAD = {"end": [0, 40, 65], "falls": [0, 40, 20], "first": [-1, 20, 64], "below": [0, 10, 20, -5, 30],
       "far below": [0, 10, 20, -2 ** 31, 30], "far above": [0, 10, 20, 2 ** 31 - 1, 30],
       "no rows": [0, 64, 70], "disorder": [32, 64, 0, 32]}


@pytest.mark.parametrize("name", list(BAD) + ["many"])
@pytest.mark.parametrize("H,Hkv,d,dt", [(2, 1, 64, "f16"), (8, 1, 128, "bf16"), (3, 3, 64, "bf16")])
def test_bad_starts_leave_the_gradients_of_other_sequences(name, H, Hkv, d, dt):
    """Valid sequences get their gradients, rows that no valid sequence owns are left alone,
    whatever the workspace held."""
    cu, T = bad_starts(700, 3) if name == "many" else (BAD[name], 64)
    B, dtype = len(cu) - 1, DT[dt]
    q, k, v, dout, _, _ = case([T], [T], H, Hkv, d, dtype, seed=T + H)
    gq, gk, gv, gd = (x.cuda() for x in (q, k, v, dout))
    o, dq = (torch.full((T, H, d), float("nan"), dtype=dtype, device="cuda") for _ in range(2))
    dk, dv = (torch.full((T, Hkv, d), float("nan"), dtype=dtype, device="cuda") for _ in range(2))
    lse = torch.full((T, H), float("nan"), device="cuda")
    size = max(fa.fa_varlen_workspace_size(B, H, Hkv, T, T, d),
               fa.fa_bwd_varlen_workspace_size(B, H, Hkv, T, T, d))
    ws = torch.full((size,), 255, dtype=torch.uint8, device="cuda")
    c, scale = i32(cu), 1 / math.sqrt(d)
    fa.fa_fwd_varlen(gq, gk, gv, o, lse, c, c, scale, ws)
    assert fa.fa_get_device_status() == fa.FA_ERR_BAD_PAGE
    ws.fill_(255)
    fa.fa_bwd_varlen(gq, gk, gv, o, gd, lse, dq, dk, dv, c, c, scale, ws)
    assert fa.fa_get_device_status() == fa.FA_ERR_BAD_PAGE
    rows = torch.ones(T, dtype=torch.bool)
    for a, b in [(a, b) for a, b in zip(cu, cu[1:]) if 0 <= a <= b <= T]:
        rows[a:b] = False
        ref = gradients(q[a:b], k[a:b], v[a:b], dout[a:b], [0, b - a], [0, b - a], scale, dtype,
                        fa.FA_MASK_CAUSAL)
        check_gradients((dq[a:b], dk[a:b], dv[a:b]), ref, b - a, b - a, f"{name} [{a}, {b})")
    for x in (dq, dk, dv):
        assert x[rows.cuda()].isnan().all()


def test_bad_starts_of_one_side_leave_the_gradients_of_other_sequences():
    H, Hkv, d, T, dtype = 4, 2, 64, 64, torch.float16
    q, k, v, dout, _, _ = case([T], [T], H, Hkv, d, dtype, seed=5)
    gq, gk, gv, gd = (x.cuda() for x in (q, k, v, dout))
    for cu_q, cu_k in (([0, 10, 20, -5, 30], [0, 12, 30, 40, 64]),
                       ([0, 12, 30, 40, 64], [0, 10, 20, -5, 30])):
        o, dq = (torch.full((T, H, d), float("nan"), dtype=dtype, device="cuda") for _ in range(2))
        dk, dv = (torch.full((T, Hkv, d), float("nan"), dtype=dtype, device="cuda")
                  for _ in range(2))
        lse = torch.full((T, H), float("nan"), device="cuda")
        size = max(fa.fa_varlen_workspace_size(4, H, Hkv, T, T, d),
                   fa.fa_bwd_varlen_workspace_size(4, H, Hkv, T, T, d))
        ws = torch.full((size,), 255, dtype=torch.uint8, device="cuda")
        fa.fa_fwd_varlen(gq, gk, gv, o, lse, i32(cu_q), i32(cu_k), 0.125, ws)
        ws.fill_(255)
        fa.fa_bwd_varlen(gq, gk, gv, o, gd, lse, dq, dk, dv, i32(cu_q), i32(cu_k), 0.125, ws)
        assert fa.fa_get_device_status() == fa.FA_ERR_BAD_PAGE
        ref = gradients(q[:cu_q[2]], k[:cu_k[2]], v[:cu_k[2]], dout[:cu_q[2]], cu_q[:3], cu_k[:3],
                        0.125, dtype, fa.FA_MASK_CAUSAL)
        check_gradients((dq, dk, dv), ref, cu_q[2], cu_k[2], f"{cu_q} {cu_k}")
        assert dk[cu_k[2]:].isnan().all() and dv[cu_k[2]:].isnan().all()


@pytest.mark.parametrize("H,Hkv,d", [(2, 1, 64), (8, 1, 128), (64, 1, 64)])
@pytest.mark.parametrize("cu", [[0, 64, 0, 64], [0, 64, 0, 64, 0, 64, 0, 64], [10, 64, 3, 60, 0, 5]],
                         ids=str)
def test_sequences_that_claim_the_same_rows_stay_in_them(H, Hkv, d, cu):
    """Reported, dk and dv of the claimed rows are finite, every other row is left alone."""
    T, B, dtype = 72, len(cu) - 1, torch.float16
    q, k, v, dout, _, _ = case([T], [T], H, Hkv, d, dtype, seed=H)
    gq, gk, gv, gd = (x.cuda() for x in (q, k, v, dout))
    o, dq = (torch.full((T, H, d), float("nan"), dtype=dtype, device="cuda") for _ in range(2))
    dk, dv = (torch.full((T, Hkv, d), float("nan"), dtype=dtype, device="cuda") for _ in range(2))
    lse = torch.full((T, H), float("nan"), device="cuda")
    size = max(fa.fa_varlen_workspace_size(B, H, Hkv, T, T, d),
               fa.fa_bwd_varlen_workspace_size(B, H, Hkv, T, T, d))
    guard = 1 << 16
    ws = torch.full((size + guard,), 255, dtype=torch.uint8, device="cuda")
    fa.fa_fwd_varlen(gq, gk, gv, o, lse, i32(cu), i32(cu), 0.125, ws[:size])
    assert fa.fa_get_device_status() == fa.FA_ERR_BAD_PAGE
    o.nan_to_num_(0.0), lse.nan_to_num_(0.0)
    ws[:size].fill_(255)
    fa.fa_bwd_varlen(gq, gk, gv, o, gd, lse, dq, dk, dv, i32(cu), i32(cu), 0.125, ws[:size])
    assert fa.fa_get_device_status() == fa.FA_ERR_BAD_PAGE
    rows = torch.zeros(T, dtype=torch.bool)
    for a, b in zip(cu, cu[1:]):
        rows[a:max(a, b)] = True
    for x in (dk, dv):
        assert x[rows.cuda()].isfinite().all()
    for x in (dq, dk, dv):
        assert x[~rows.cuda()].isnan().all()
    assert (ws[size:] == 255).all()
