"""Rotary positions through the C ABI against a plain implementation in 64 bits.

Tolerance: cos and sin are off by at most about 2^-22 (the angle's fraction of a turn rounded to
FP32, then sincospif), the two products and their sum add three FP32 roundings, and the result is
rounded once to its type: |dy| <= (u + 2^-20) A (|x_a| + |x_b|), with u = eps / 2 (fp32: u is
already below the 2^-20)."""
import pytest
import torch

import tiled_attention_06_gb300 as fa

from _packed import half_step, rotate, starts

pytestmark = pytest.mark.gpu

DT = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(scope="module", autouse=True)
def _built():
    from tiled_attention_06_gb300 import build
    build.build()
    fa.lib()


def draw(shape, dtype, seed):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed)).to(dtype)


def limit(x, rot, half, amplitude, dtype):
    """The bound on every element, from the magnitudes of its pair."""
    a = x.double().abs()
    lim = a.clone() * 0
    if half:
        s = a[..., :rot // 2] + a[..., rot // 2:rot]
        lim[..., :rot // 2], lim[..., rot // 2:rot] = s, s
    else:
        s = a[..., 0:rot:2] + a[..., 1:rot:2]
        lim[..., 0:rot:2], lim[..., 1:rot:2] = s, s
    return lim * abs(amplitude) * (half_step(dtype) + 2.0 ** -20) + 2.0 ** -24


def check(x, pos, freqs, rot, style, amplitude=1.0, inverse=False, in_place=False):
    dev = "cuda"
    xg = x.to(dev)
    y = xg if in_place else torch.full_like(xg, float("nan"))
    fa.fa_rope(xg, y, pos.to(dev), freqs.to(dev), style, amplitude, inverse)
    half = style == fa.FA_ROPE_HALF
    ref = rotate(x, pos, freqs, rot, half, amplitude, inverse)
    got = y.double().cpu()
    err = (got - ref).abs()
    lim = limit(x, rot, half, amplitude, x.dtype)
    assert (err <= lim).all(), float((err - lim).max())
    assert torch.equal(got[..., rot:], x.double()[..., rot:])  # the rest passes through
    return y


@pytest.mark.parametrize("style", [fa.FA_ROPE_HALF, fa.FA_ROPE_PAIRS])
@pytest.mark.parametrize("dt", list(DT))
@pytest.mark.parametrize("T,H,d,rot", [(1, 1, 64, 64), (3, 5, 128, 128), (700, 2, 128, 64),
                                       (65, 3, 96, 34), (5, 2, 6, 4), (2, 1, 512, 512),
                                       (2500, 40, 128, 128)])
def test_rotation_and_its_inverse(T, H, d, rot, dt, style):
    x = draw((T, H, d), DT[dt], seed=T + d)
    pos = torch.randint(0, 5000, (T,), generator=torch.Generator().manual_seed(3),
                        dtype=torch.int32)
    freqs, amp = fa.fa_rope_freqs(rot)
    assert amp == 1.0
    check(x, pos, freqs, rot, style)
    check(x, pos, freqs, rot, style, inverse=True, in_place=True)


@pytest.mark.parametrize("pos", [0, -1, 2 ** 31 - 1, -2 ** 31, 1000003])
def test_far_positions_keep_their_angle(pos):
    """pos * w reaches 2^31 rad; the reference's 64-bit product is itself off by 2^-22 there."""
    freqs, _ = fa.fa_rope_freqs(128)
    x = draw((2, 3, 128), torch.float32, seed=1)
    p = torch.full((2,), pos, dtype=torch.int32)
    y = torch.empty_like(x, device="cuda")
    fa.fa_rope(x.cuda(), y, p.cuda(), freqs.cuda())
    err = (y.double().cpu() - rotate(x, p, freqs, 128, True)).abs()
    a = x.double().abs()
    s = a[..., :64] + a[..., 64:]
    lim = torch.cat([s, s], -1) * (2.0 ** -20 + abs(pos) * 2.0 ** -53) + 2.0 ** -24
    assert (err <= lim).all(), float((err - lim).max())


def test_zero_and_unit_frequencies_and_amplitude():
    x = draw((4, 2, 64), torch.float32, seed=2)
    pos = torch.tensor([0, 1, 2, 3], dtype=torch.int32)
    freqs = torch.zeros(32, dtype=torch.float64)
    freqs[1] = -1.5
    freqs[2] = 2 * torch.pi
    check(x, pos, freqs, 64, fa.FA_ROPE_HALF, amplitude=1.25)


@pytest.mark.parametrize("style", [fa.FA_ROPE_HALF, fa.FA_ROPE_PAIRS])
def test_strides_and_misaligned_views(style):
    """q and k as slices of a fused projection, head-major views, a view that starts off 16
    bytes, and rows around the view left as they were."""
    freqs, _ = fa.fa_rope_freqs(64)
    fg = freqs.cuda()
    base = draw((37, 9, 64), torch.bfloat16, seed=4)
    pos = torch.arange(37, dtype=torch.int32) * 11
    for view in (lambda t: t[:, 2:7], lambda t: t[3:30, :1], lambda t: t.transpose(0, 1)[:, 5:20]):
        x = view(base)
        p = pos[:x.shape[0]]
        out = torch.full_like(base, 7.0).cuda()
        fa.fa_rope(view(base.cuda()), view(out), p.cuda(), fg, style)
        want = rotate(x, p, freqs, 64, style == fa.FA_ROPE_HALF)
        lim = limit(x, 64, style == fa.FA_ROPE_HALF, 1.0, torch.bfloat16)
        got = out.cpu()
        assert ((view(got).double() - want).abs() <= lim).all()
        view(got).fill_(7.0)
        assert (got == 7.0).all()
    flat = draw((1 + 20 * 3 * 64,), torch.float16, seed=5)
    odd = flat[1:].view(20, 3, 64)
    buf = torch.zeros(1 + 20 * 3 * 64, dtype=torch.float16, device="cuda")
    y = buf[1:].view(20, 3, 64)
    src = flat.cuda()[1:].view(20, 3, 64)
    fa.fa_rope(src, y, pos[:20].cuda(), fg, style)
    want = rotate(odd, pos[:20], freqs, 64, style == fa.FA_ROPE_HALF)
    lim = limit(odd, 64, style == fa.FA_ROPE_HALF, 1.0, torch.float16)
    assert ((y.double().cpu() - want).abs() <= lim).all()


def test_inverse_is_the_gradient_by_differences():
    """<dy, R(x + h e) - R(x - h e)> / 2h = (R^T dy)_e: the map is linear, so the difference has
    no truncation error and the FP32 roundings (2^-22 of sums of 2 terms over h = 1) remain."""
    freqs, _ = fa.fa_rope_freqs(16)
    fg, pos = freqs.cuda(), torch.tensor([9], dtype=torch.int32, device="cuda")
    dy = draw((1, 1, 16), torch.float32, seed=6).cuda()
    dx = torch.empty_like(dy)
    fa.fa_rope(dy, dx, pos, fg, fa.FA_ROPE_PAIRS, 1.5, True)
    for e in range(16):
        x = torch.zeros(1, 1, 16, device="cuda")
        x[0, 0, e] = 1.0
        up, down = torch.empty_like(x), torch.empty_like(x)
        fa.fa_rope(x, up, pos, fg, fa.FA_ROPE_PAIRS, 1.5)
        fa.fa_rope(-x, down, pos, fg, fa.FA_ROPE_PAIRS, 1.5)
        d = float((dy * (up - down)).double().sum()) / 2
        assert abs(d - float(dx[0, 0, e])) <= 2.0 ** -18 * (1 + float(dy.abs().max()))


# ------------------------------------------------------------------ rotate and append

def cache(B, Hkv, page, d, width, pages, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    table = torch.randperm(pages, generator=g)[:B * width].reshape(B, width).to(torch.int32)
    kp = torch.full((pages, Hkv, page, d), float("nan"), dtype=dtype)
    return table, kp, kp.clone()


@pytest.mark.parametrize("style", [fa.FA_ROPE_HALF, fa.FA_ROPE_PAIRS])
@pytest.mark.parametrize("H,Hkv,d,rot,page,dt", [(8, 2, 128, 128, 16, "bf16"),
                                                 (3, 3, 64, 32, 64, "f16"),
                                                 (7, 1, 128, 50, 256, "bf16")])
def test_append_writes_the_new_slots_alone(H, Hkv, d, rot, page, dt, style):
    new, before = [1, 0, 37, 5, 1], [0, 12, page - 3, 2 * page, page - 1]
    B, width, pages, dtype = len(new), 5, 40, DT[dt]
    T, cu = sum(new), starts(new)
    pad = 2  # rows behind the last sequence
    qkv = draw((T + pad, H + 2 * Hkv, d), dtype, seed=8)
    table, kp, vp = cache(B, Hkv, page, d, width, pages, dtype, seed=9)
    freqs, amp = fa.fa_rope_freqs(rot, scaling=fa.FA_ROPE_BY_PARTS, factor=4.0, trained_len=2048)
    kg, vg = kp.cuda(), vp.cuda()
    out = torch.full((T + pad, H, d), 3.0, dtype=dtype, device="cuda")
    x = qkv.cuda()
    ctx = torch.tensor(before, dtype=torch.int32).cuda()
    fa.fa_rope_append(x[:, :H], x[:, H:H + Hkv], x[:, H + Hkv:], out, kg, vg, table.cuda(), ctx,
                      torch.tensor(cu, dtype=torch.int32).cuda(), freqs.cuda(), style, amp)
    assert fa.fa_get_device_status() == fa.FA_OK
    half = style == fa.FA_ROPE_HALF
    got, k_got, v_got = out.cpu(), kg.cpu(), vg.cpu()
    written = torch.zeros(pages, page, dtype=torch.bool)
    for b in range(B):
        rows = slice(cu[b], cu[b + 1])
        pos = torch.arange(before[b], before[b] + new[b])
        for name, src, have in (("q", qkv[rows, :H], got[rows]),
                                ("k", qkv[rows, H:H + Hkv], None)):
            want = rotate(src, pos, freqs, rot, half, amp)
            if have is None:
                have = k_got[table[b, pos // page].long(), :, pos % page]
            lim = limit(src, rot, half, amp, dtype)
            assert ((have.double() - want).abs() <= lim).all(), (name, b)
        slots = v_got[table[b, pos // page].long(), :, pos % page]
        assert torch.equal(slots, qkv[rows, H + Hkv:])
        written[table[b, pos // page].long(), pos % page] = True
    assert (got[T:] == 3.0).all()
    for pool in (k_got, v_got):
        assert pool.transpose(1, 2)[~written].isnan().all()
        assert not pool.transpose(1, 2)[written].isnan().any()


def test_append_reports_and_skips_bad_slots():
    H, Hkv, d, page = 2, 1, 64, 16
    qkv = draw((4, H + 2 * Hkv, d), torch.float16, seed=1).cuda()
    kp = torch.zeros(3, Hkv, page, d, dtype=torch.float16, device="cuda")
    vp = kp.clone()
    table = torch.tensor([[5, -1], [1, 2]], dtype=torch.int32, device="cuda")
    ctx = torch.tensor([3, 31], dtype=torch.int32, device="cuda")  # 31 + 2 is over 2 pages
    cu = torch.tensor([0, 2, 4], dtype=torch.int32, device="cuda")
    freqs, _ = fa.fa_rope_freqs(d, device="cuda")
    out = torch.zeros(4, H, d, dtype=torch.float16, device="cuda")
    fa.fa_rope_append(qkv[:, :H], qkv[:, H:H + 1], qkv[:, H + 1:], out, kp, vp, table, ctx, cu,
                      freqs)
    assert fa.fa_get_device_status() == fa.FA_ERR_BAD_PAGE
    assert fa.fa_get_device_status() == fa.FA_OK
    assert (kp[0] == 0).all() and (kp[1] == 0).all()
    assert torch.equal(vp[2, :, 15], qkv[2, H + 1:])  # position 31 is the last slot
    assert (vp[2, :, :15] == 0).all()
    assert (out != 0).any(-1).all()  # every q is rotated


@pytest.mark.parametrize("style", [fa.FA_ROPE_HALF, fa.FA_ROPE_PAIRS])
def test_append_of_many_sequences(style):
    """More sequences than a CTA has threads, and CTAs whose tokens belong to several of them."""
    H, Hkv, d, page, B, dtype = 2, 1, 64, 16, 901, torch.bfloat16
    new, before = [(3 * b) % 8 for b in range(B)], [(5 * b) % 30 for b in range(B)]
    T, cu = sum(new), starts(new)
    assert T > 16 * 152  # several tokens per CTA
    width, pages = 3, B * 3
    qkv = draw((T, H + 2 * Hkv, d), dtype, seed=11)
    table = torch.randperm(pages, generator=torch.Generator().manual_seed(2)).reshape(B, width)
    kg, vg = (torch.full((pages, Hkv, page, d), float("nan"), dtype=dtype, device="cuda")
              for _ in range(2))
    freqs, amp = fa.fa_rope_freqs(d)
    x = qkv.cuda()
    out = torch.full((T, H, d), float("nan"), dtype=dtype, device="cuda")
    args = (x[:, :H], x[:, H:H + Hkv], x[:, H + Hkv:], out, kg, vg, table.to(torch.int32).cuda(),
            torch.tensor(before, dtype=torch.int32).cuda(),
            torch.tensor(cu, dtype=torch.int32).cuda(), freqs.cuda(), style, amp)
    graph = torch.cuda.CUDAGraph()  # once captured, once by itself: the same bits
    with torch.cuda.graph(graph):
        fa.fa_rope_append(*args)
    graph.replay()
    torch.cuda.synchronize()
    first = [t.clone() for t in (out, kg, vg)]
    fa.fa_rope_append(*args)
    assert fa.fa_get_device_status() == fa.FA_OK
    for a, b in zip(first, (out, kg, vg)):
        assert torch.equal(a.view(torch.int16), b.view(torch.int16))
    seq = torch.repeat_interleave(torch.arange(B), torch.tensor(new))
    pos = torch.tensor(before)[seq] + torch.arange(T) - torch.tensor(cu)[seq]
    at = (table[seq, pos // page], slice(None), pos % page)
    half = style == fa.FA_ROPE_HALF
    for src, have in ((qkv[:, :H], out.cpu()), (qkv[:, H:H + Hkv], kg.cpu()[at])):
        err = (have.double() - rotate(src, pos, freqs, d, half, amp)).abs()
        assert (err <= limit(src, d, half, amp, dtype)).all()
    assert torch.equal(vg.cpu()[at], qkv[:, H + Hkv:])
    assert int((~vg.isnan()).any(-1).sum()) == T * Hkv


BAD = {"end": lambda T: [0, 40, T + 1], "falls": lambda T: [0, 40, 20],
       "first": lambda T: [-1, 20, T], "below": lambda T: [0, 10, 20, -5, T],
       "far below": lambda T: [0, 10, 20, -2 ** 31, T],
       "far above": lambda T: [0, 10, 20, 2 ** 31 - 1, T], "no rows": lambda T: [0, T, T + 6],
       "disorder": lambda T: [40, T, 0, 40]}


@pytest.mark.parametrize("name", list(BAD) + ["many"])
@pytest.mark.parametrize("long", [False, True])
def test_append_reports_bad_starts_and_keeps_other_sequences(name, long):
    """Valid sequences are rotated and cached, no other token writes anything; for one token
    per CTA and for several."""
    H, Hkv, d, page, dtype = 2, 1, 64, 16, torch.float16
    T = 16 * torch.cuda.get_device_properties(0).multi_processor_count + 3 if long else 64
    if name == "many":
        g = torch.Generator().manual_seed(4)
        cu = starts(torch.randint(0, 8 if long else 2, (700,), generator=g).tolist())
        T = max(cu[-1], T)
        cu[0] = cu[233] = cu[660] = -9
        cu[350] = T + 50
        cu[175], cu[176] = 3, T + 9
    else:
        cu = BAD[name](T)
    B = len(cu) - 1
    good = [(b, cu[b], cu[b + 1]) for b in range(B) if 0 <= cu[b] <= cu[b + 1] <= T]
    before = [(7 * b) % 20 for b in range(B)]
    width = (20 + T) // page + 1
    # pages of a sequence's own, and one for all that it must not reach
    need = {b: -(-(before[b] + e - a) // page) for b, a, e in good}
    table = torch.zeros(B, width, dtype=torch.int32)
    at = 1
    for b, n in need.items():
        table[b, :n] = torch.arange(at, at + n)
        at += n
    qkv = draw((T, H + 2 * Hkv, d), dtype, seed=21)
    freqs, amp = fa.fa_rope_freqs(d)
    kg, vg = (torch.full((at, Hkv, page, d), float("nan"), dtype=dtype, device="cuda")
              for _ in range(2))
    out = torch.full((T, H, d), float("nan"), dtype=dtype, device="cuda")
    x = qkv.cuda()
    fa.fa_rope_append(x[:, :H], x[:, H:H + Hkv], x[:, H + Hkv:], out, kg, vg, table.cuda(),
                      torch.tensor(before, dtype=torch.int32).cuda(),
                      torch.tensor(cu, dtype=torch.int32).cuda(), freqs.cuda())
    assert fa.fa_get_device_status() == fa.FA_ERR_BAD_PAGE
    assert fa.fa_get_device_status() == fa.FA_OK
    got, kc, vc = out.cpu(), kg.cpu(), vg.cpu()
    rows = torch.ones(T, dtype=torch.bool)
    written = torch.zeros(at, page, dtype=torch.bool)
    for b, a, e in good:
        rows[a:e] = False
        pos = before[b] + torch.arange(e - a)
        slot = (table[b, pos // page].long(), slice(None), pos % page)
        written[slot[0], slot[2]] = True
        for src, have in ((qkv[a:e, :H], got[a:e]), (qkv[a:e, H:H + Hkv], kc[slot])):
            err = (have.double() - rotate(src, pos, freqs, d, True, amp)).abs()
            assert (err <= limit(src, d, True, amp, dtype)).all(), (b, a, e)
        assert torch.equal(vc[slot], qkv[a:e, H + Hkv:])
    assert got[rows].isnan().all()
    for pool in (kc, vc):
        assert pool.transpose(1, 2)[~written].isnan().all()


def test_append_beyond_32_bit_positions():
    """A chunk whose positions pass 2^31: nothing of it is cached, its q is rotated."""
    H, d, page = 2, 64, 16
    qkv = draw((3, H + 2, d), torch.float16, seed=2).cuda()
    kp = torch.zeros(2, 1, page, d, dtype=torch.float16, device="cuda")
    vp = kp.clone()
    freqs, _ = fa.fa_rope_freqs(d)
    out = torch.full((3, H, d), float("nan"), dtype=torch.float16, device="cuda")
    ints = [torch.tensor(x, dtype=torch.int32, device="cuda")
            for x in ([[0, 1]], [2 ** 31 - 2], [0, 3])]
    fa.fa_rope_append(qkv[:, :H], qkv[:, H:H + 1], qkv[:, H + 1:], out, kp, vp, *ints, freqs.cuda())
    assert fa.fa_get_device_status() == fa.FA_ERR_BAD_PAGE
    pos = 2 ** 31 - 2 + torch.arange(3)
    x = qkv[:, :H].cpu()
    err = (out.double().cpu() - rotate(x, pos, freqs, d, True)).abs()
    # the reference's own 64-bit product and the frequencies' fixed point: 2^-21 rad
    lim = limit(x, d, True, 1.0, torch.float16) * (1 + 2.0 ** -9)
    assert (err <= lim).all(), float((err - lim).max())
    assert (kp == 0).all() and (vp == 0).all()
