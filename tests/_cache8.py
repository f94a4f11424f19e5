"""Plain 64-bit forms of the norm with a rotation, its gradient and the 8-bit cache, with bounds.

Norm and rotation. Between load and store everything is FP32: the sum of d squares is off by at
most (16 + 5) 2^-24 of itself, 1/sqrt by 2^-22, sine and cosine by 2^-22, and the angle as a float
fraction of a turn by pi 2^-24, so a rotated element is off by less than 2^-19 (|n_a| + |n_b|)
before its one rounding. The gradient has one product and one mean more: 2^-18 of the sums of
magnitudes. A weight's gradient adds a thread's rows one by one (below 64 here): 2^-17 of them.

8 bits. An element is at most half a step of its own binade off, in units of its row's power, plus
what the FP32 value was off. The power itself is the exact one unless the row's largest magnitude is
within 2^-18 of a border. Rows copied from 16 bits (V) have neither error: equal bytes.
"""
import torch

import _packed as ref
import tiled_attention_06_gb300 as fa


def pair_bound(n, rot, half):
    """|n_a| + |n_b| for both elements of a pair, |n| for the rest."""
    r = n.abs().clone()
    if half:
        a, b = slice(0, rot // 2), slice(rot // 2, rot)
    else:
        a, b = slice(0, rot, 2), slice(1, rot, 2)
    both = n[..., a].abs() + n[..., b].abs()
    r[..., a] = both
    r[..., b] = both
    return r


def turn(x, pos, axis, freqs, rot, half, amplitude=1.0, inverse=False):
    """x [T, H, d] in 64 bits, pos [axes, T]."""
    y = x.double().clone()
    t = (pos.double()[axis.long()].T * freqs.double()[None])[:, None] * (-1 if inverse else 1)
    c, s = t.cos() * amplitude, t.sin() * amplitude
    if half:
        a, b = slice(0, rot // 2), slice(rot // 2, rot)
    else:
        a, b = slice(0, rot, 2), slice(1, rot, 2)
    u, v = x.double()[..., a], x.double()[..., b]
    y[..., a] = u * c - v * s
    y[..., b] = v * c + u * s
    return y


def normed(x, w, eps):
    """x / sqrt(mean(x^2) + eps) * w; eps None: x."""
    x = x.double()
    if eps is None:
        return x
    n = x / (x.square().mean(-1, keepdim=True) + eps).sqrt()
    return n if w is None else n * w.double()


def norm_rope(x, w, eps, pos, axis, freqs, rot, half, amplitude=1.0):
    """(y, bound on the FP32 error) in 64 bits."""
    n = normed(x, w, eps)
    y = turn(n, pos, axis, freqs, rot, half, amplitude)
    return y, 2.0 ** -19 * max(1.0, abs(amplitude)) * pair_bound(n, rot, half)


def norm_rope_grad(x, w, eps, dy, pos, axis, freqs, rot, half, amplitude=1.0):
    """(dx, bound), (dw, bound) in 64 bits."""
    g = turn(dy, pos, axis, freqs, rot, half, amplitude, inverse=True)
    big = max(1.0, abs(amplitude)) * pair_bound(dy.double(), rot, half)
    if eps is None:
        return (g, 2.0 ** -19 * big), None
    x = x.double()
    w = torch.ones(x.shape[-1], dtype=torch.float64) if w is None else w.double()
    r = 1 / (x.square().mean(-1, keepdim=True) + eps).sqrt()
    dx = r * w * g - x * r ** 3 * (w * g * x).mean(-1, keepdim=True)
    e = r * w.abs() * big + x.abs() * r ** 3 * (w.abs() * big * x.abs()).mean(-1, keepdim=True)
    dw = (g * x * r).sum((0, 1))
    return (dx, 2.0 ** -18 * e), (dw, 2.0 ** -17 * (big * x.abs() * r).sum((0, 1)))


def check(got, want, bound, dtype, what):
    got = got.double().cpu()
    assert torch.isfinite(got).all(), f"{what}: non-finite"
    over = (got - want).abs() - bound - ref.half_step(dtype) * (want.abs() + bound) - 2.0 ** -25
    assert (over <= 0).all(), f"{what}: {float(over.max()):.3e} over its bound"


# ------------------------------------------------------------------------------ 8 bits

def exponent_byte(amax):
    """The smallest byte in [0, 254] with amax <= 448 * 2^(byte - 127) (float64 in)."""
    m, e = torch.frexp(amax)
    e = torch.where(m > 0.875, e - 8, e - 9)
    return torch.where(amax == 0, -127, e).clamp(-127, 127).to(torch.int64) + 127


def quantise(x):
    """x [..., d] -> (bytes uint8, exponent bytes uint8); 64 bits inside."""
    x = x.double()
    bad = ~torch.isfinite(x).all(-1)
    x = torch.where(bad[..., None], torch.zeros((), dtype=torch.float64), x)
    b = exponent_byte(x.abs().amax(-1))
    y = x * torch.exp2(127.0 - b.double())[..., None]
    _, e = torch.frexp(y)
    step = torch.exp2((e.clamp(min=-5) - 4).double())  # smallest binade: 2^-6, step 2^-9
    y = (y / step).round() * step  # to nearest, ties to even
    return y.float().to(torch.float8_e4m3fn).view(torch.uint8), \
        torch.where(bad, 255, b).to(torch.uint8)


def values(bytes8, exponents):
    """What the rows stand for, float64."""
    x = bytes8.view(torch.float8_e4m3fn).float().double()
    p = torch.exp2(exponents.double() - 127)
    return x * torch.where(exponents == 255, float("nan"), p)[..., None]


def half_steps(y, exponents):
    """Half a step of the cache at the value y of a row."""
    p = torch.exp2(exponents.double() - 127)[..., None]
    _, e = torch.frexp(y / p)
    return torch.exp2((e.clamp(min=-5) - 5).double()) * p


class Cache:
    """A pool whose pages are taken in random order, on the CPU; every unused slot holds garbage."""

    def __init__(self, ctx, Hkv, d, page, seed=0, bits=8, dtype=torch.bfloat16, rows=None):
        g = torch.Generator().manual_seed(seed)
        need = [-(-c // page) for c in ctx]
        P = sum(need) + 2
        order = torch.randperm(P, generator=g).tolist()
        width = max(max(need), 1) + 1
        self.table = torch.full((len(ctx), width), -1, dtype=torch.int32)
        at = 0
        for b, k in enumerate(need):
            self.table[b, :k] = torch.tensor(order[at:at + k], dtype=torch.int32)
            at += k
        self.page, self.bits, self.dtype = page, bits, dtype
        make = rows or (lambda *s: torch.randn(*s, d, generator=g) *
                        torch.exp(0.5 * torch.randn(*s, 1, generator=g)))
        self.pages, self.scales = [], []
        for _ in range(2):
            x = make(P, Hkv, page)
            if bits == 8:
                q, e = quantise(x)
                self.pages.append(q)
                self.scales.append(e)
            else:
                self.pages.append(x.to(dtype))
        used = torch.zeros(P, page, dtype=torch.bool)
        for b, c in enumerate(ctx):
            for i in range(need[b]):
                used[self.table[b, i], :max(0, min(page, c - i * page))] = True
        gone = ~used[:, None].expand(P, Hkv, page)
        for i in range(2):
            if bits == 8:
                self.pages[i][gone] = 0x7f
                self.scales[i][gone] = 255
            else:
                self.pages[i][gone] = float("nan")

    def rows(self, b, n):
        """(k, v) of the first n positions of sequence b, [n, Hkv, d] float64."""
        p = self.table[b, :-(-n // self.page)].long()
        out = []
        for i in range(2):
            x = values(self.pages[i][p], self.scales[i][p]) if self.bits == 8 else \
                self.pages[i][p].double()
            out.append(x.transpose(1, 2).flatten(0, 1)[:n])
        return out

    def cuda(self):
        """(pools and table, dict of the exponents)"""
        k, v = (x.cuda() for x in self.pages)
        kw = {}
        if self.bits == 8:
            k, v = k.view(torch.float8_e4m3fn), v.view(torch.float8_e4m3fn)
            kw = {n: e.cuda().view(torch.float8_e8m0fnu)
                  for n, e in zip(("k_scales", "v_scales"), self.scales)}
        return (k, v, self.table.cuda()), kw


def trees(lengths, words, seed=0, blank=()):
    """int32 [sum + 2, words] of random trees; tokens in `blank` (packed rows) see none. Bits behind
    a chunk's end are set: they have to be ignored."""
    g = torch.Generator().manual_seed(seed)
    rows = []
    for n in lengths:
        seen = []
        for j in range(n):
            up = int(torch.randint(-1, j, (1,), generator=g)) if j else -1
            seen.append((seen[up] if up >= 0 else 0) | 1 << j)
        rows += [s | ((1 << 32 * words) - (1 << n)) for s in seen]
    rows = [0 if i in blank else r for i, r in enumerate(rows)] + [0, 0]
    words_of = [[(r >> 32 * w) & 0xffffffff for w in range(words)] for r in rows]
    return torch.tensor(words_of, dtype=torch.int64).to(torch.int32)


def tree_seen(tree, first, n, m):
    """[n, m] bool of one sequence whose tokens are the packed rows from `first` on."""
    vis = torch.ones(n, m, dtype=torch.bool)
    for i in range(n):
        for j in range(n):
            at = m - n + j
            if at >= 0:
                vis[i, at] = bool((int(tree[first + i, j // 32]) >> (j % 32)) & 1)
    return vis


def attention(q, cache, ctx, lengths, scale, mask, window=0, n_global=0, tree=None):
    """o, lse and the bound on |o - o_ref| without u, as _packed.attention."""
    T, H, d = q.shape
    o = torch.zeros(T, H, d, dtype=torch.float64)
    lse = torch.zeros(T, H, dtype=torch.float64)
    bound = torch.zeros(T, H, dtype=torch.float64)
    at = 0
    for b, (n, m) in enumerate(zip(lengths, ctx)):
        k, v = cache.rows(b, m)
        G = H // k.shape[1] if m else 1
        vis = tree_seen(tree, at, n, m) if tree is not None else \
            ref.seen(n, m, mask, window, n_global)
        for h in range(H):
            if m == 0:
                lse[at:at + n, h] = float("-inf")
                continue
            p, oh, l = ref.head(q[at:at + n, h], k[:, h // G], v[:, h // G], vis, scale)
            o[at:at + n, h], lse[at:at + n, h] = oh, l
            big = v[:, h // G].abs().amax(-1)
            bound[at:at + n, h] = (vis * big[None]).amax(-1) if n else 0
        at += n
    return o, lse, bound
