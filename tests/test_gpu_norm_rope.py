"""Norms of query and key heads with rotary positions, their gradient, the form that writes a cache in
16 and 8 bits, and the 8-bit cache read back, against the formulas in 64 bits."""
import math

import pytest
import torch

import _cache8 as c8
import _packed as ref
import tiled_attention_06_gb300 as fa

pytestmark = pytest.mark.gpu
BF, HF, FP = torch.bfloat16, torch.float16, torch.float32


def status_ok():
    torch.cuda.synchronize()
    assert fa.fa_get_device_status() == fa.FA_OK


def randn(*shape, dtype=FP, seed=0):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed)).to(dtype)


def axis_of(rot, axes):
    n = rot // 2
    sections = [n // axes + (1 if a < n % axes else 0) for a in range(axes)]
    return fa.fa_rope_axes(sections, interleaved=axes % 2 == 0)


CASES = [  # T, H, Hkv, d, rot, axes, half, dtype, weights' dtype (None: none), eps (None: no norm)
    (1, 4, 1, 64, 64, 1, True, BF, BF, 1e-6),
    (5, 3, 2, 128, 128, 3, True, HF, FP, 1e-5),
    (70, 8, 2, 128, 64, 2, False, BF, BF, 1e-6),
    (33, 2, 1, 64, 30, 3, True, HF, HF, 1e-6),     # element by element
    (9, 5, 1, 80, 80, 4, False, BF, None, 1e-6),   # five units: an odd number of lanes
    (12, 2, 2, 256, 192, 3, True, BF, BF, 0.1),
    (3, 1, 1, 512, 512, 1, False, HF, FP, 1e-6),
    (7, 2, 0, 2, 2, 1, True, BF, BF, 1e-6),
    (11, 3, 1, 512, 256, 2, True, FP, FP, 1e-6),
    (65, 4, 2, 64, 64, 4, False, FP, FP, 1e-6),
    (17, 1, 3, 6, 4, 1, False, FP, None, 1e-3),
    (40, 6, 2, 128, 128, 3, True, BF, None, None),
    (2500, 3, 1, 64, 64, 3, True, BF, BF, 1e-6),   # several tokens per CTA
    (2433, 1, 1, 16, 8, 1, False, HF, HF, 1e-6),
]


class Problem:
    def __init__(self, case, seed=0):
        T, H, Hkv, d, rot, axes, half, dtype, wdt, eps = case
        self.case, self.rot, self.half, self.eps = case, rot, half, eps
        qkv = randn(T, H + 2 * Hkv + 1, d, dtype=dtype, seed=seed)
        self.qkv = qkv.cuda()
        self.x = [qkv[:, :H], qkv[:, H:H + Hkv]]
        self.dev = [self.qkv[:, :H], self.qkv[:, H:H + Hkv]]
        g = torch.Generator().manual_seed(seed + 1)
        self.pos = torch.randint(-(1 << 31), (1 << 31) - 1, (axes, T), generator=g, dtype=torch.int64)
        self.pos[:, : (T + 1) // 2] %= 3000
        self.pos = self.pos.to(torch.int32)
        self.axis = axis_of(rot, axes) if axes > 1 else torch.zeros(rot // 2, dtype=torch.int32)
        # frequencies that are exact fractions of a turn leave the 64-bit reference exact as well
        k = torch.randint(1, 1 << 20, (rot // 2,), generator=g)
        self.freqs = k.double() / (1 << 32) * 2 * math.pi
        self.w = [None if wdt is None else (1 + 0.3 * randn(d, seed=seed + 2 + i)).to(wdt)
                  for i in range(2)]
        self.amp = 1.25
        self.kw = dict(style=fa.FA_ROPE_HALF if half else fa.FA_ROPE_PAIRS, amplitude=self.amp,
                       pair_axis=self.axis.cuda() if axes > 1 else None)
        if eps is not None:
            self.kw.update(norm=fa.FA_NORM_RMS, eps=eps, q_weight=self._c(0), k_weight=self._c(1))

    def _c(self, i):
        return None if self.w[i] is None else self.w[i].cuda()

    def angles(self):
        """Positions that the reference can turn in 64 bits: modulo the frequencies' period."""
        return self.pos.double() % float(1 << 32)


def reference_angles(p):
    """sin and cos see the position modulo 2^32 turns of the unit 2^-32: exact in 64 bits."""
    return p.angles()


@pytest.mark.parametrize("case", CASES, ids=str)
def test_norm_rope(case):
    p = Problem(case)
    T, H, Hkv, d, rot, axes, half, dtype, wdt, eps = case
    out = [torch.full((T + 1, n, d), 7.0, dtype=dtype, device="cuda") for n in (H, Hkv)]
    fa.fa_norm_rope(p.dev[0], p.dev[1] if Hkv else None, out[0][:T], out[1][:T] if Hkv else None,
                    p.pos.cuda(), p.freqs.cuda(), **p.kw)
    status_ok()
    for i, n in enumerate((H, Hkv)):
        if not n:
            continue
        y, bound = c8.norm_rope(p.x[i], p.w[i], eps, reference_angles(p), p.axis, p.freqs, rot, half,
                                p.amp)
        c8.check(out[i][:T], y, bound, dtype, "qk"[i])
        assert (out[i][T] == 7).all()


@pytest.mark.parametrize("case", CASES, ids=str)
def test_norm_rope_gradient(case):
    p = Problem(case, seed=5)
    T, H, Hkv, d, rot, axes, half, dtype, wdt, eps = case
    dy = [randn(T, n, d, dtype=dtype, seed=20 + n) for n in (H, Hkv)]
    dx = torch.full((T, H + Hkv + 1, d), 7.0, dtype=dtype, device="cuda")
    dw = [torch.full((d,), 7.0, device="cuda") for _ in range(2)]
    kw = dict(p.kw)
    if eps is not None:
        kw.update(dq_weight=dw[0], dk_weight=dw[1], workspace=torch.empty(
            fa.fa_norm_rope_bwd_workspace_size(H, Hkv, d), dtype=torch.uint8, device="cuda"))
    args = [p.dev[0], p.dev[1] if Hkv else None, dy[0].cuda(), dy[1].cuda() if Hkv else None,
            dx[:, :H], dx[:, H:H + Hkv] if Hkv else None, p.pos.cuda(), p.freqs.cuda()]
    fa.fa_norm_rope_bwd(*args, **kw)
    status_ok()
    for i, at in enumerate((slice(0, H), slice(H, H + Hkv))):
        if at.start == at.stop:
            assert eps is None or (dw[i] == 0).all()  # a sum over nothing
            continue
        (gx, bx), gw = c8.norm_rope_grad(p.x[i], p.w[i], eps, dy[i], reference_angles(p), p.axis,
                                         p.freqs, rot, half, p.amp)
        c8.check(dx[:, at], gx, bx, dtype, "d" + "qk"[i])
        if gw is not None:
            c8.check(dw[i], gw[0], gw[1], FP, "dw" + "qk"[i])
    assert (dx[:, H + Hkv] == 7).all()
    again = [x.clone() for x in (dx, *dw)]
    fa.fa_norm_rope_bwd(*args, **kw)
    assert all(torch.equal(a, b) for a, b in zip(again, (dx, *dw)))  # the same bits


SPREAD = [  # heads over several CTAs, long runs of tokens per CTA, the last of them ragged
    (7, 80, 8, 128, 128, 3, True, BF, BF, 1e-6),
    (5, 33, 7, 256, 256, 2, False, HF, FP, 1e-6),
    (3, 23, 9, 512, 512, 1, True, BF, BF, 1e-6),
    (2, 700, 5, 64, 32, 1, False, BF, BF, 1e-6),
    (2, 50, 1, 198, 66, 2, True, FP, FP, 1e-6),     # element by element
    (20011, 2, 1, 64, 64, 2, True, BF, BF, 1e-6),
    (15013, 1, 1, 34, 30, 1, False, HF, HF, 1e-6),
    (9001, 1, 0, 16, 16, 4, True, FP, FP, 1e-6),
]


@pytest.mark.parametrize("case", SPREAD, ids=str)
def test_many_heads_and_many_tokens(case):
    test_norm_rope(case)
    test_norm_rope_gradient(case)


CHUNKS = [  # rotated parts that end inside 16 bytes, rows of three, five and six lanes
    (45, 6, 2, 128, 66, 1, False, BF, BF, 1e-6),
    (45, 6, 2, 128, 66, 1, True, BF, BF, 1e-6),
    (31, 3, 1, 64, 40, 2, True, HF, HF, 1e-6),
    (31, 3, 1, 64, 36, 2, True, BF, FP, 1e-6),
    (31, 3, 1, 64, 38, 3, False, HF, HF, 1e-6),
    (26, 4, 2, 64, 20, 1, True, FP, FP, 1e-6),
    (26, 4, 2, 64, 22, 1, False, FP, FP, 1e-6),
    (26, 4, 2, 64, 22, 1, True, FP, FP, 1e-6),
    (300, 8, 2, 80, 80, 3, True, BF, BF, 1e-6),
    (301, 7, 3, 96, 96, 1, False, HF, HF, 1e-6),
    (77, 7, 3, 96, 2, 1, True, BF, BF, 1e-6),
    (1203, 5, 1, 48, 48, 1, True, BF, BF, 1e-6),
    (50, 2, 1, 256, 250, 1, False, BF, BF, 1e-6),
    (50, 2, 1, 80, 76, 4, True, FP, FP, 1e-6),
    (9, 41, 7, 80, 18, 2, False, BF, BF, 1e-6),
]


@pytest.mark.parametrize("case", CHUNKS, ids=str)
def test_chunks_and_groups(case):
    test_norm_rope(case)
    test_norm_rope_gradient(case)


def test_elements_behind_the_rotated_part_are_copied():
    T, H, d, rot = 6, 2, 64, 38
    x = randn(T, H, d, dtype=BF, seed=1)
    x[:, :, rot:] = torch.tensor([float("inf"), -0.0, float("-inf"), 1.0])[torch.arange(d - rot) % 4].to(BF)
    freqs = fa.fa_rope_freqs(rot)[0].cuda()
    for style in (fa.FA_ROPE_HALF, fa.FA_ROPE_PAIRS):
        y = torch.empty_like(x).cuda()
        fa.fa_norm_rope(x.cuda(), None, y, None, torch.arange(T, dtype=torch.int32).cuda(), freqs,
                        style=style)
        status_ok()
        assert torch.equal(y[:, :, rot:].cpu().view(torch.int16), x[:, :, rot:].view(torch.int16))
        assert torch.isfinite(y[:, :, :rot]).all()


def test_gradients_on_two_streams_and_of_one_weight():
    """Own workspaces, and either weight's gradient alone: the same as one after the other."""
    T, H, Hkv, d = 600, 6, 2, 128
    freqs, pos = fa.fa_rope_freqs(d)[0].cuda(), torch.arange(T, dtype=torch.int32).cuda()
    streams = [torch.cuda.Stream() for _ in range(3)]
    runs = []
    for i, s in enumerate([None] * 3 + streams):
        i %= 3
        x = [randn(T, n, d, dtype=BF, seed=i + n).cuda() for n in (H, Hkv)]
        dy = [randn(T, n, d, dtype=BF, seed=10 + i + n).cuda() for n in (H, Hkv)]
        w = [(1 + 0.1 * randn(d, seed=i + n)).cuda() for n in range(2)]
        dx, dw = [torch.empty_like(t) for t in x], [torch.full((d,), 7.0, device="cuda") for _ in w]
        ws = torch.empty(fa.fa_norm_rope_bwd_workspace_size(H, Hkv, d), dtype=torch.uint8, device="cuda")
        runs.append((x, dy, dx, w, dw, ws, s, i))
    torch.cuda.synchronize()
    for _ in range(3):
        for x, dy, dx, w, dw, ws, s, i in runs:
            fa.fa_norm_rope_bwd(*x, *dy, *dx, pos, freqs, *w, dw[0] if i != 1 else None,
                                dw[1] if i != 2 else None, ws, norm=fa.FA_NORM_RMS, stream=s)
    status_ok()
    for a, b in zip(runs[:3], runs[3:]):
        assert all(torch.equal(u, v) for u, v in zip(a[2] + a[4], b[2] + b[4]))
    assert (runs[1][4][0] == 7).all() and (runs[2][4][1] == 7).all()


def test_gradient_against_differences():
    """A step of 2^-9 in 32 bits along a random direction: the difference quotient's own error is
    its third derivative (below 2^-12 here) and FP32 noise over the step (2^-22 * 2^9)."""
    T, H, d = 6, 2, 64
    x, g, v = (randn(T, H, d, seed=i).cuda() for i in (1, 2, 3))
    w, dwt = (1 + 0.2 * randn(d, seed=4)).cuda(), randn(d, seed=5).cuda()
    pos = torch.arange(T, dtype=torch.int32, device="cuda")
    freqs = fa.fa_rope_freqs(d)[0].cuda()

    def f(x, w):
        y = torch.empty_like(x)
        fa.fa_norm_rope(x, None, y, None, pos, freqs, q_weight=w, norm=fa.FA_NORM_RMS, eps=1e-6)
        return (y.double() * g.double()).sum().item()

    dx, dw = torch.empty_like(x), torch.empty(d, device="cuda")
    ws = torch.empty(fa.fa_norm_rope_bwd_workspace_size(H, 0, d), dtype=torch.uint8, device="cuda")
    fa.fa_norm_rope_bwd(x, None, g, None, dx, None, pos, freqs, q_weight=w, dq_weight=dw,
                        workspace=ws, norm=fa.FA_NORM_RMS, eps=1e-6)
    h = 2.0 ** -9
    for got, a, b in (((dx.double() * v.double()).sum().item(), f(x + h * v, w), f(x - h * v, w)),
                      ((dw.double() * dwt.double()).sum().item(), f(x, w + h * dwt), f(x, w - h * dwt))):
        assert abs((a - b) / (2 * h) - got) <= 2.0 ** -8 * (1 + abs(got)), (got, (a - b) / (2 * h))


@pytest.mark.parametrize("size", [1e-15, 1e-18, 1e15])
def test_rows_far_from_one(size):
    """Lengths whose cube leaves 32 bits, without an eps to hold them: the same directions."""
    T, H, d = 5, 2, 64
    x = (randn(T, H, d, seed=1) * size).to(BF)
    dy = randn(T, H, d, dtype=BF, seed=2)
    w = (1 + 0.2 * randn(d, seed=3)).to(BF)
    pos, freqs = torch.arange(T, dtype=torch.int32), fa.fa_rope_freqs(d)[0]
    args = (pos[None], torch.zeros(d // 2), freqs, d, True)
    y, dx = (torch.empty(T, H, d, dtype=BF, device="cuda") for _ in range(2))
    dw = torch.empty(d, device="cuda")
    ws = torch.empty(fa.fa_norm_rope_bwd_workspace_size(H, 0, d), dtype=torch.uint8, device="cuda")
    kw = dict(q_weight=w.cuda(), norm=fa.FA_NORM_RMS, eps=0.0)
    fa.fa_norm_rope(x.cuda(), None, y, None, pos.cuda(), freqs.cuda(), **kw)
    fa.fa_norm_rope_bwd(x.cuda(), None, dy.cuda(), None, dx, None, pos.cuda(), freqs.cuda(),
                        dq_weight=dw, workspace=ws, **kw)
    status_ok()
    want, bound = c8.norm_rope(x, w, 0.0, *args)
    c8.check(y, want, bound, BF, "y")
    (gx, bx), (gw, bw) = c8.norm_rope_grad(x, w, 0.0, dy, *args)
    scale = 2.0 ** round(math.log2(float(gx.abs().max())))  # exact in both
    c8.check(dx.double() / scale, gx / scale, bx / scale, BF, "dx")
    c8.check(dw, gw, bw, FP, "dw")


def test_in_place_and_head_major_layouts():
    T, H, d = 37, 4, 64
    x = randn(H, T, d, dtype=BF, seed=3)  # [heads, tokens, d]
    pos = torch.arange(T, dtype=torch.int32)
    freqs = fa.fa_rope_freqs(d)[0]
    view = x.cuda().transpose(0, 1)
    want, bound = c8.norm_rope(x.transpose(0, 1), None, 1e-6, pos[None], torch.zeros(d // 2), freqs,
                               d, True)
    fa.fa_norm_rope(view, None, view, None, pos.cuda(), freqs.cuda(), norm=fa.FA_NORM_RMS, eps=1e-6)
    c8.check(view, want, bound, BF, "in place")
    # gradients in place of the upstream ones
    dy = randn(H, T, d, dtype=BF, seed=4)
    view = dy.cuda().transpose(0, 1)
    q = x.cuda().transpose(0, 1)
    fa.fa_norm_rope_bwd(q, None, view, None, view, None, pos.cuda(), freqs.cuda(),
                        norm=fa.FA_NORM_RMS, eps=1e-6)
    (gx, bx), _ = c8.norm_rope_grad(x.transpose(0, 1), None, 1e-6, dy.transpose(0, 1), pos[None],
                                    torch.zeros(d // 2), freqs, d, True)
    c8.check(view, gx, bx, BF, "gradient in place")


def test_unaligned_rows_take_the_element_path():
    T, H, d = 9, 3, 64
    flat = randn(T * H * d + 1, dtype=BF, seed=6).cuda()
    x = flat[1:].view(T, H, d)
    y = torch.empty(T * H * d + 1, dtype=BF, device="cuda")[1:].view(T, H, d)
    z = torch.empty(T, H, d, dtype=BF, device="cuda")
    pos = torch.arange(T, dtype=torch.int32, device="cuda")
    freqs = fa.fa_rope_freqs(d)[0].cuda()
    kw = dict(norm=fa.FA_NORM_RMS, eps=1e-6)
    fa.fa_norm_rope(x, None, y, None, pos, freqs, **kw)
    fa.fa_norm_rope(x.clone(), None, z, None, pos, freqs, **kw)
    # the sums' orders differ: a rounding may fall the other way, by one step
    assert ((y.double() - z.double()).abs() <= 2.0 ** -7 * z.double().abs()).all()
    assert (y != z).double().mean() < 0.01


def test_no_tokens_zeroes_the_weights_gradients():
    d = 64
    e = torch.empty(0, 2, d, dtype=BF, device="cuda")
    dw = [torch.ones(d, device="cuda") for _ in range(2)]
    pos = torch.empty(1, 0, dtype=torch.int32, device="cuda")
    freqs = fa.fa_rope_freqs(d)[0].cuda()
    ws = torch.empty(fa.fa_norm_rope_bwd_workspace_size(2, 2, d), dtype=torch.uint8, device="cuda")
    fa.fa_norm_rope(e, e, e, e, pos, freqs, norm=fa.FA_NORM_RMS)
    fa.fa_norm_rope_bwd(e, e, e, e, e, e, pos, freqs, dq_weight=dw[0], dk_weight=dw[1], workspace=ws,
                        norm=fa.FA_NORM_RMS)
    status_ok()
    assert all((w == 0).all() for w in dw)


def test_axis_out_of_range_is_reported_and_read_as_the_first():
    T, d = 4, 64
    x = randn(T, 1, d, dtype=BF).cuda()
    pos = torch.arange(2 * T, dtype=torch.int32, device="cuda").view(2, T)
    freqs = fa.fa_rope_freqs(d)[0].cuda()
    axis = torch.zeros(d // 2, dtype=torch.int32, device="cuda")
    y, z = torch.empty_like(x), torch.empty_like(x)
    fa.fa_norm_rope(x, None, y, None, pos, freqs, pair_axis=axis)
    status_ok()
    axis[3], axis[4] = 2, -1
    fa.fa_norm_rope(x, None, z, None, pos, freqs, pair_axis=axis)
    torch.cuda.synchronize()
    assert fa.fa_get_device_status() == fa.FA_ERR_BAD_PAGE
    assert torch.equal(y, z)


def test_captured_gradient_follows_its_inputs():
    T, H, Hkv, d = 30, 4, 2, 128
    x = [randn(T, n, d, dtype=BF, seed=n).cuda() for n in (H, Hkv)]
    dy = [randn(T, n, d, dtype=BF, seed=9 + n).cuda() for n in (H, Hkv)]
    dx = [torch.empty_like(t) for t in x]
    w = [(1 + 0.1 * randn(d, seed=i)).to(BF).cuda() for i in range(2)]
    dw = [torch.empty(d, device="cuda") for _ in range(2)]
    pos = torch.arange(T, dtype=torch.int32, device="cuda")
    freqs = fa.fa_rope_freqs(d)[0].cuda()
    ws = torch.empty(fa.fa_norm_rope_bwd_workspace_size(H, Hkv, d), dtype=torch.uint8, device="cuda")

    def step():
        fa.fa_norm_rope_bwd(*x, *dy, *dx, pos, freqs, *w, *dw, ws, norm=fa.FA_NORM_RMS)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for t in x + dy:
        t.copy_(torch.randn_like(t))
    pos.add_(17)
    ws.fill_(255)
    graph.replay()
    got = [t.clone() for t in dx + dw]
    step()
    status_ok()
    assert all(torch.equal(a, b) for a, b in zip(got, dx + dw))


# ------------------------------------------------------------------------------ into the cache

APPENDS = [  # lengths, cached before, H, Hkv, d, rot, page, axes (0: places), half, dtype, bits, norm
    ([1] * 5, [0, 15, 16, 17, 300], 4, 1, 64, 64, 16, 0, True, BF, 8, True),
    ([3, 0, 70, 1], [5, 9, 60, 0], 3, 3, 128, 128, 64, 3, True, HF, 8, True),
    ([40, 2], [0, 255], 8, 2, 128, 50, 256, 2, False, BF, 8, True),
    ([17], [1000], 2, 2, 64, 32, 48, 4, False, HF, 8, False),
    ([3, 0, 70, 1], [5, 9, 60, 0], 3, 3, 128, 128, 64, 3, True, HF, 16, True),
    ([900, 1600], [100, 3], 2, 1, 64, 64, 128, 0, False, BF, 8, True),
    ([20, 20], [7, 40], 4, 2, 128, 128, 16, 0, True, BF, 16, False),
]


class Append:
    def __init__(self, case, seed=0):
        lens, before, H, Hkv, d, rot, page, axes, half, dtype, bits, norm = case
        T = sum(lens)
        self.T, self.lens, self.before = T, lens, before
        self.cu = torch.tensor(ref.starts(lens), dtype=torch.int32)
        qkv = randn(T + 2, H + 2 * Hkv, d, seed=seed) * torch.exp(randn(T + 2, H + 2 * Hkv, 1, seed=seed + 1))
        self.qkv = qkv.to(dtype)
        self.split = [slice(0, H), slice(H, H + Hkv), slice(H + Hkv, H + 2 * Hkv)]
        self.cache = c8.Cache([b + n for b, n in zip(before, lens)], Hkv, d, page, seed, bits, dtype)
        place = torch.cat([torch.arange(b, b + n) for b, n in zip(before, lens)])
        g = torch.Generator().manual_seed(seed + 2)
        self.pos = torch.randint(0, 4000, (axes, T + 2), generator=g) if axes else None
        self.angles = place[None] if axes == 0 else self.pos[:, :T]
        self.axis = axis_of(rot, axes) if axes > 1 else torch.zeros(rot // 2, dtype=torch.int32)
        self.freqs = fa.fa_rope_freqs(rot)[0]
        self.w = [(1 + 0.2 * randn(d, seed=seed + 3 + i)).to(dtype) if norm else None for i in range(2)]
        self.eps = 1e-6 if norm else None
        self.place = place

    def call(self, pools, kw, q_out, qkv=None, stream=None):
        lens, before, H, Hkv, d, rot, page, axes, half, dtype, bits, norm = self.case
        dev = self.qkv.cuda() if qkv is None else qkv
        if norm:
            kw = dict(kw, norm=fa.FA_NORM_RMS, eps=1e-6, q_weight=self.w[0].cuda(),
                      k_weight=self.w[1].cuda())
        fa.fa_norm_rope_append(
            *[dev[:, s] for s in self.split], q_out, *pools,
            torch.tensor(before, dtype=torch.int32).cuda(), self.cu.cuda(), self.freqs.cuda(),
            positions=None if self.pos is None else self.pos.to(torch.int32).cuda(),
            pair_axis=self.axis.cuda() if axes > 1 else None,
            style=fa.FA_ROPE_HALF if half else fa.FA_ROPE_PAIRS, stream=stream, **kw)


@pytest.mark.parametrize("case", APPENDS, ids=str)
def test_append(case):
    a = Append(case)
    a.case = case
    lens, before, H, Hkv, d, rot, page, axes, half, dtype, bits, norm = case
    T = a.T
    pools, kw = a.cache.cuda()
    was = [x.clone() for x in pools[:2]] + [x.clone() for x in kw.values()]
    q_out = torch.full((T + 2, H, d), 7.0, dtype=dtype, device="cuda")
    a.call(pools, kw, q_out)
    status_ok()
    args = (a.angles, a.axis, a.freqs, rot, half)
    y, bound = c8.norm_rope(a.qkv[:T, a.split[0]], a.w[0], a.eps, *args)
    c8.check(q_out[:T], y, bound, dtype, "q")
    assert (q_out[T:] == 7).all()
    seq = torch.cat([torch.full((n,), b) for b, n in enumerate(lens)])
    at = a.cache.table[seq, a.place // page].long(), slice(None), a.place % page
    k, kb = c8.norm_rope(a.qkv[:T, a.split[1]], a.w[1], a.eps, *args)
    v = a.qkv[:T, a.split[2]]
    now = [x.cpu() for x in pools[:2]] + [x.cpu() for x in kw.values()]
    if bits == 16:
        c8.check(now[0][at], k, kb, dtype, "k")
        assert torch.equal(now[1][at], v)
    else:
        kq, vq, ke, ve = (x.view(torch.uint8)[at] for x in now)
        want, power = c8.quantise(v)
        assert torch.equal(vq, want) and torch.equal(ve, power)
        exact = c8.exponent_byte(k.abs().amax(-1))
        border = c8.exponent_byte(k.abs().amax(-1) * (1 + 2.0 ** -18)) != \
            c8.exponent_byte(k.abs().amax(-1) * (1 - 2.0 ** -18))
        assert ((ke.long() == exact) | border).all()
        lim = c8.half_steps(k.abs() + kb, ke) * (1 + 2.0 ** -10) + kb
        assert ((c8.values(kq, ke) - k).abs() <= lim).all()
    # nothing else was written
    for x, y in zip(now, was):
        x, y = x.view(torch.uint8).clone(), y.cpu().view(torch.uint8).clone()
        x[at] = 0
        y[at] = 0
        assert torch.equal(x, y)


def test_append_of_rows_that_cannot_be_scaled():
    """Zeros, an infinity, a NaN, the largest and the smallest rows of V."""
    d, page = 64, 16
    v = torch.zeros(7, 1, d)
    v[1, 0, 3], v[2, 0, 9] = float("inf"), float("nan")
    v[3], v[4], v[5], v[6] = 3e38, 448.0, 450.0, 1e-40
    v = v.to(BF)
    q = torch.ones(7, 1, d, dtype=BF)
    pages = [torch.full((2, 1, page, d), 9, dtype=torch.uint8, device="cuda") for _ in range(2)]
    scales = [torch.full((2, 1, page), 9, dtype=torch.uint8, device="cuda") for _ in range(2)]
    i32 = dict(dtype=torch.int32, device="cuda")
    table, zero, cu = torch.tensor([[1]], **i32), torch.tensor([0], **i32), torch.tensor([0, 7], **i32)
    fa.fa_norm_rope_append(q.cuda(), q.cuda(), v.cuda(), q.cuda(), *pages, table, zero, cu,
                           fa.fa_rope_freqs(d)[0].cuda(), k_scales=scales[0], v_scales=scales[1])
    status_ok()
    want, power = c8.quantise(v)
    got = scales[1][1, 0, :7].cpu()
    assert torch.equal(got, power[:, 0])
    assert got.tolist()[:5] == [0, 255, 255, 247, 127] and got[5] == 128
    assert torch.equal(pages[1][1, 0, :7].cpu(), want[:, 0])
    out = [torch.empty(7, 1, d, dtype=BF, device="cuda") for _ in range(2)]
    fa.fa_kv_read(*pages, *scales, table, zero, cu, *out)
    status_ok()
    back = out[1].cpu()
    assert back[1:3].isnan().all() and torch.isfinite(back[[0, 3, 4, 5]]).all()
    assert (back[0] == 0).all() and (back[4] == 448).all() and (back[5] == 448).all()


def test_append_with_bad_pages_and_starts():
    """A token without a slot keeps its q, others keep everything; bad starts own nothing."""
    case = ([3, 4, 2], [0, 14, 5], 2, 1, 64, 64, 16, 0, True, BF, 8, True)
    a = Append(case)
    a.case = case
    a.cache.table[1, 1] = 1000  # positions 16 and 17 of the second sequence
    pools, kw = a.cache.cuda()
    q_out = torch.full((a.T + 2, 2, 64), 7.0, dtype=BF, device="cuda")
    a.call(pools, kw, q_out)
    torch.cuda.synchronize()
    assert fa.fa_get_device_status() == fa.FA_ERR_BAD_PAGE
    y, bound = c8.norm_rope(a.qkv[:a.T, a.split[0]], a.w[0], 1e-6, a.angles, a.axis, a.freqs, 64, True)
    c8.check(q_out[:a.T], y, bound, BF, "q")
    want, power = c8.quantise(a.qkv[:a.T, a.split[2]])
    vp, vs = pools[1].view(torch.uint8).cpu(), kw["v_scales"].view(torch.uint8).cpu()
    for t, (b, p) in {0: (0, 0), 1: (0, 1), 2: (0, 2), 3: (1, 14), 4: (1, 15), 7: (2, 5), 8: (2, 6)}.items():
        page = a.cache.table[b, p // 16]
        assert torch.equal(vp[page, 0, p % 16], want[t, 0]) and vs[page, 0, p % 16] == power[t, 0]
    a.cu = torch.tensor([0, 3, 2, 9], dtype=torch.int32)  # the second starts behind its end
    q_out.fill_(7)
    a.call(pools, kw, q_out)
    torch.cuda.synchronize()
    assert fa.fa_get_device_status() == fa.FA_ERR_BAD_PAGE
    assert torch.isfinite(q_out[:2].float()).all() and (q_out[a.T:] == 7).all()


@pytest.mark.parametrize("rot,half", [(66, True), (66, False), (40, True), (36, True), (72, False)])
@pytest.mark.parametrize("bits", [8, 16])
def test_append_of_rotated_parts_that_end_inside_16_bytes(rot, half, bits):
    test_append(([3, 0, 70, 1], [5, 9, 60, 0], 6, 3, 128, rot, 64, 3, half, HF, bits, True))


@pytest.mark.parametrize("bits", [8, 16])
def test_append_for_many_sequences_and_heads(bits):
    """More sequences than a CTA has threads; heads over several CTAs; several batches of tokens."""
    test_append(([1, 0, 2] * 300, [3, 40, 17] * 300, 2, 1, 64, 64, 16, 0, True, BF, bits, True))
    test_append(([5, 30], [9, 2], 70, 10, 128, 128, 64, 3, True, HF, bits, True))
    test_append(([6000, 1, 5000], [3, 200, 0], 1, 1, 64, 64, 256, 2, False, BF, bits, True))


# ------------------------------------------------------------------------------ read back

@pytest.mark.parametrize("lens,starts,Hkv,d,page,dtype", [
    ([1, 0, 5], [0, 3, 15], 1, 64, 16, BF), ([300, 17], [1, 250], 2, 128, 64, HF),
    ([64], [64], 3, 128, 48, BF), ([1, 0, 3] * 400, [7, 0, 20] * 400, 2, 64, 16, BF), ([3000, 8000, 1], [5, 0, 77], 1, 64, 256, HF)], ids=str)
def test_read(lens, starts, Hkv, d, page, dtype):
    ctx = [n + s for n, s in zip(lens, starts)]
    cache = c8.Cache(ctx, Hkv, d, page, seed=3)
    (k, v, table), kw = cache.cuda()
    T = sum(lens)
    wide = torch.full((T + 1, 3 * Hkv, d), 7.0, dtype=dtype, device="cuda")
    cu = torch.tensor(ref.starts(lens), dtype=torch.int32).cuda()
    fa.fa_kv_read(k, v, kw["k_scales"], kw["v_scales"], table,
                  torch.tensor(starts, dtype=torch.int32).cuda(), cu, wide[:, :Hkv], wide[:, Hkv:2 * Hkv])
    status_ok()
    got, at = wide.cpu(), 0
    for b, (n, s) in enumerate(zip(lens, starts)):
        for i, x in enumerate(cache.rows(b, n + s)):
            assert torch.equal(got[at:at + n, i * Hkv:(i + 1) * Hkv], x[s:].to(dtype))
        at += n
    assert (got[T] == 7).all() and (got[:, 2 * Hkv:] == 7).all()


def test_read_of_bad_pages_gives_zeros():
    cache = c8.Cache([40, 20], 1, 64, 16, seed=1)
    cache.table[0, 1] = -5
    (k, v, table), kw = cache.cuda()
    i32 = dict(dtype=torch.int32, device="cuda")
    out = [torch.full((60, 1, 64), 7.0, dtype=BF, device="cuda") for _ in range(2)]
    fa.fa_kv_read(k, v, kw["k_scales"], kw["v_scales"], table, torch.tensor([0, 0], **i32),
                  torch.tensor([0, 40, 60], **i32), *out)
    torch.cuda.synchronize()
    assert fa.fa_get_device_status() == fa.FA_ERR_BAD_PAGE
    for i in range(2):
        got = out[i].cpu()
        assert (got[16:32] == 0).all()
        cache.table[0, 1] = 0
        want = cache.rows(0, 40)[i].to(BF)
        assert torch.equal(got[:16], want[:16]) and torch.equal(got[32:40], want[32:])
        assert torch.equal(got[40:], cache.rows(1, 20)[i].to(BF))
        cache.table[0, 1] = -5
