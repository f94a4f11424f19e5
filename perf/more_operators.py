"""Norms of query and key heads with a rotation of several axes (and their gradient), the same step
written into an 8-bit cache, that cache read back, attention over it, and attention of trees of
drafted tokens over a cache: the cases they are measured on, their plain form in elementary torch
operations, and the framework's calls.

Layouts: tokens are packed, [tokens, heads, d]; sequence b owns the rows cu[b] .. cu[b+1]-1.
Pools are [num_pages, kv_heads, page, d] with an int32 block table per sequence; query head h
reads K/V head h // (H // Hkv). A row of an 8-bit cache (one token and head) is d values of 4
exponent and 3 mantissa bits times one power of two, whose exponent takes a byte of its own.
"""
import math
import random

import torch

own = False

DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
MOST_SCORES = 8 * 32 * 512 * 8192  # padded scores of the largest listed case
MOST_KEYS = 32 * 8192 * 8          # padded keys times K/V heads of the largest listed case
PAD = 3                            # rows behind the last sequence that belong to nobody


# ------------------------------------------------------------------------------ cases

def listed():
    return [
        # one step of 64 sequences: the query and key heads of the fused projection
        dict(name="norm_step", op="norm", T=64, H=32, Hkv=8, d=128, rot=128, style="half", axes=1,
             order="blocks", norm=True, dtype="bf16", max_pos=1 << 20),
        # the prompts of a batch with images among the text: time, height and width
        dict(name="norm_prompt", op="norm", T=16384, H=32, Hkv=8, d=128, rot=128, style="half",
             axes=3, order="blocks", norm=True, dtype="bf16", max_pos=8192),
        # a training step's gradient, text alone
        dict(name="grad_train", op="grad", T=16384, H=32, Hkv=8, d=128, rot=128, style="half",
             axes=1, order="blocks", norm=True, dtype="bf16", max_pos=8192),
        # the same for video, half of a small head rotated as neighbours, axes taking turns, odd
        # number of tokens
        dict(name="grad_odd", op="grad", T=8191, H=16, Hkv=4, d=64, rot=32, style="pairs", axes=3,
             order="turns", norm=True, dtype="f16", max_pos=4096),
        # one new token for each of 64 sequences into the cache
        dict(name="append_step", op="append", B=64, H=32, Hkv=8, d=128, rot=128, style="half",
             axes=1, order="blocks", norm=True, dtype="bf16", page=256, max_ctx=2048, max_new=1,
             lens_seed=1),
        # ragged chunks of up to 512 tokens of eight sequences, image positions, 64-token pages
        dict(name="append_chunk", op="append", B=8, H=32, Hkv=8, d=128, rot=128, style="half",
             axes=3, order="blocks", norm=True, dtype="f16", page=64, max_ctx=8192, max_new=512,
             lens_seed=2),
        # prefixes of a chat batch, read back to be shared
        dict(name="read_short", op="read", B=16, H=8, Hkv=8, d=128, dtype="f16", page=64,
             max_ctx=512, max_new=256, lens_seed=3),
        # whole contexts read back
        dict(name="read_long", op="read", B=16, H=8, Hkv=8, d=128, dtype="bf16", page=256,
             max_ctx=8192, max_new=8192, lens_seed=4),
        # one token per sequence over contexts of up to 8192 tokens
        dict(name="cache_step", op="cache", B=32, H=32, Hkv=8, d=128, mask="causal", window=0,
             bits=8, dtype="bf16", page=256, max_ctx=8192, min_new=1, max_new=1, lens_seed=5),
        # chunks of a prompt next to what is cached of it
        dict(name="cache_chunk", op="cache", B=8, H=32, Hkv=8, d=128, mask="causal", window=0,
             bits=8, dtype="bf16", page=256, max_ctx=8192, min_new=1, max_new=512, lens_seed=6),
        # trees of 32 drafted tokens checked at once, 16-bit cache
        dict(name="tree_wide", op="cache", B=8, H=32, Hkv=8, d=128, mask="tree", window=0, bits=16,
             dtype="bf16", page=64, max_ctx=16384, min_new=32, max_new=32, lens_seed=7),
        # small trees over long contexts in 8 bits
        dict(name="tree_small", op="cache", B=4, H=16, Hkv=8, d=128, mask="tree", window=0, bits=8,
             dtype="f16", page=64, max_ctx=65536, min_new=1, max_new=7, lens_seed=8),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["norm", "grad", "append", "read", "cache", "cache", "cache"])
    hkv = rng.choice([1, 2, 3, 4, 8])
    H = hkv * rng.choice([1, 2, 3, 4, 5, 7, 8])
    d = rng.choice([64, 128])
    dtype = rng.choice(["f16", "bf16", "bf16"])
    axes = rng.choice([1, 1, 2, 3, 4])
    rope = dict(rot=d if rng.random() < 0.5 else 2 * rng.randint(2, d // 2),
                style=rng.choice(["half", "pairs"]), axes=axes,
                order=rng.choice(["blocks", "turns"]), norm=rng.random() < 0.8)
    if op in ("norm", "grad"):
        d = rng.choice([64, 80, 96, 128, 256])
        rope["rot"] = min(rope["rot"], d)
        return dict(op=op, T=_log(rng, 1, 16384 if d <= 128 else 8192), H=min(H, 32), Hkv=hkv, d=d,
                    dtype=rng.choice(["f16", "bf16", "bf16", "f32"]) if d <= 64 else dtype,
                    max_pos=_log(rng, 16, 1 << 20), **rope)
    seed = rng.randrange(1 << 30)
    page = rng.choice([16, 64, 128, 256])
    if op == "append":
        return dict(op=op, B=_log(rng, 1, 64), H=H, Hkv=hkv, d=d, dtype=dtype, page=page,
                    max_ctx=_log(rng, 600, 2048), max_new=_log(rng, 1, 256), lens_seed=seed, **rope)
    B, ctx = _log(rng, 1, 64), _log(rng, 64, 32768)
    if op == "read":
        while B * ctx * hkv > MOST_KEYS // 2:
            B, ctx = max(1, B * 3 // 4), max(64, ctx * 7 // 8)
        return dict(op=op, B=B, H=hkv, Hkv=hkv, d=d, dtype=dtype, page=page, max_ctx=ctx,
                    max_new=_log(rng, 1, ctx), lens_seed=seed)
    mask = rng.choice(["causal", "causal", "window", "tree", "tree"])
    bits = 16 if mask == "tree" and rng.random() < 0.5 else 8
    new = _log(rng, 1, 128) if mask == "tree" else rng.choice([1, 1, _log(rng, 1, 512)])
    while B * ctx * hkv > MOST_KEYS or B * H * new * ctx > MOST_SCORES:
        B, ctx, new = max(1, B * 3 // 4), max(64, ctx * 7 // 8), max(1, new * 7 // 8)
    return dict(op=op, B=B, H=H, Hkv=hkv, d=d, mask=mask,
                window=_log(rng, 1, 2048) if mask == "window" else 0, bits=bits, dtype=dtype,
                page=page, max_ctx=ctx, min_new=1, max_new=min(new, ctx), lens_seed=seed)


def _lengths(case):
    """(tokens, tokens cached before them) of every sequence."""
    rng = random.Random(case["lens_seed"])
    out = []
    for _ in range(case["B"]):
        n = rng.randint(case.get("min_new", 1), case["max_new"])
        total = rng.randint(n, max(n, case["max_ctx"]))
        out.append((n, total - n))
    return out


def _visible_pairs(case, n, before):
    """Visible (query, key) pairs of one sequence and head (of a tree: at most)."""
    w = case["window"] if case["mask"] == "window" else n + before
    full = max(0, min(n, w - before))  # queries that see every earlier key
    return full * before + full * (full + 1) // 2 + (n - full) * w


def work(case):
    d, H, Hkv, op = case["d"], case["H"], case["Hkv"], case["op"]
    e = 4 if case["dtype"] == "f32" else 2
    if op in ("norm", "grad"):
        n, angles = case["T"] * (H + Hkv), case["T"] * case["axes"] * 4 + case["rot"] // 2 * 8
        if op == "norm":
            return {"bytes": 2 * n * d * e + angles, "flops": n * (4 * d + 3 * case["rot"])}
        reads = 3 if case["norm"] else 2  # without a norm the gradient does not need the input
        return {"bytes": reads * n * d * e + angles, "flops": n * (10 * d + 3 * case["rot"])}
    lens = _lengths(case)
    T = sum(n for n, _ in lens)
    if op == "append":
        return {"bytes": T * d * ((2 * H + 2 * Hkv) * e + 2 * Hkv) + T * 2 * Hkv,
                "flops": T * ((H + Hkv) * (4 * d + 3 * case["rot"]) + 2 * Hkv * 2 * d)}
    if op == "read":
        return {"bytes": T * 2 * Hkv * (d * (1 + e) + 1), "flops": T * 2 * Hkv * d}
    keys = sum(min(n + c, case["window"] + n - 1) if case["mask"] == "window" else n + c
               for n, c in lens)
    row = d + 1 if case["bits"] == 8 else d * e
    return {"bytes": keys * 2 * Hkv * row + T * 2 * H * d * e + T * H * 4,
            "flops": 4 * d * H * sum(_visible_pairs(case, n, c) for n, c in lens)}


# ------------------------------------------------------------------------------ inputs

def _frequencies(case):
    """Radians per position of every rotated pair, and the axis whose position turns it."""
    n = case["rot"] // 2
    i = torch.arange(n, device="cuda")
    w = 10000.0 ** (-2.0 * i.double() / case["rot"])
    axis = i % case["axes"] if case["order"] == "turns" else i * case["axes"] // n
    return w, axis.to(torch.int32)


def _pages(case, lens, seed):
    """Block table over a pool whose pages are taken in random order, and the pool's size."""
    need = [-(-(n + c) // case["page"]) for n, c in lens]
    pool = sum(need) + 3
    order = torch.randperm(pool, generator=torch.Generator().manual_seed(int(seed) + 7)).tolist()
    width = max(need) + 1
    table = [[-1] * width for _ in lens]
    at = 0
    for b, k in enumerate(need):
        table[b][:k] = order[at:at + k]
        at += k
    return torch.tensor(table, dtype=torch.int32, device="cuda"), pool


def _trees(case, lens, seed):
    """int32 words [tokens, words]: bit j of a token's row is set where it sees token j of its own
    tree: its ancestors and itself."""
    rng = random.Random(int(seed) + 13)
    words = -(-max(n for n, _ in lens) // 32)
    rows = []
    for n, _ in lens:
        seen = []
        for j in range(n):
            up = rng.randint(-1, j - 1) if rng.random() < 0.5 else j - 1
            seen.append((seen[up] if up >= 0 else 0) | 1 << j)
        rows += [[(s >> 32 * w) & 0xffffffff for w in range(words)] for s in seen]
    rows += [[0] * words for _ in range(PAD)]
    return torch.tensor(rows, dtype=torch.int64).to(torch.int32).cuda()


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    dt, d, H, Hkv, op = DTYPES[case["dtype"]], case["d"], case["H"], case["Hkv"], case["op"]

    def randn(*shape):
        return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32)

    def spread(*shape):  # rows of different sizes, as keys and values have
        return randn(*shape, d) * torch.exp(0.5 * randn(*shape, 1))

    s = {"case": case, "H": H, "Hkv": Hkv, "scale": 1.0 / math.sqrt(d), "eps": 1e-6}
    if op in ("norm", "grad", "append"):
        s["freqs"], s["axis"] = _frequencies(case)
        s["norm"] = case["norm"]
        s["q_weight"], s["k_weight"] = ((1 + 0.1 * randn(d)).to(dt) for _ in range(2))
    i32 = dict(dtype=torch.int32, device="cuda")
    if op in ("norm", "grad"):
        T = case["T"]
        s["pos"] = torch.randint(0, case["max_pos"], (case["axes"], T), generator=g, **i32)
        qkv = randn(T, H + 2 * Hkv, d).to(dt)  # the fused projection; v is not touched
        s["q"], s["k"] = qkv[:, :H], qkv[:, H:H + Hkv]
        if op == "norm":
            out = torch.zeros(T, H + Hkv, d, dtype=dt, device="cuda")
            s["q_out"], s["k_out"] = out[:, :H], out[:, H:]
        else:
            s["dq_out"], s["dk_out"] = randn(T, H, d).to(dt), randn(T, Hkv, d).to(dt)
            s["dqkv"] = torch.zeros(T, H + 2 * Hkv, d, dtype=dt, device="cuda")
            s["dq"], s["dk"] = s["dqkv"][:, :H], s["dqkv"][:, H:H + Hkv]
            s["dq_weight"], s["dk_weight"] = (torch.zeros(d, device="cuda") for _ in range(2))
        return s
    lens = _lengths(case)
    new, before = [n for n, _ in lens], [c for _, c in lens]
    T = sum(new)
    s["cu"] = torch.tensor([sum(new[:b]) for b in range(len(new) + 1)], **i32)
    s["before"] = torch.tensor(before, **i32)
    s["ctx"] = torch.tensor([n + c for n, c in lens], **i32)
    s["max_new"], s["max_ctx"] = max(new), max(n + c for n, c in lens)
    s["table"], pool = _pages(case, lens, seed)
    for x in ("k", "v"):
        rows = spread(pool, Hkv, case["page"])
        if case.get("bits", 8) == 8:
            s[x + "_pages"], s[x + "_scales"] = _plain_quantise(rows)
        else:
            s[x + "_pages"], s[x + "_scales"] = rows.to(dt), None
        del rows
    if op == "read":
        s["k_rows"], s["v_rows"] = (torch.zeros(T + PAD, Hkv, d, dtype=dt, device="cuda")
                                    for _ in range(2))
        return s
    qkv = spread(T + PAD, H + 2 * Hkv).to(dt)
    s["q"], s["k"], s["v"] = qkv[:, :H], qkv[:, H:H + Hkv], qkv[:, H + Hkv:]
    s["o"] = torch.zeros(T + PAD, H, d, dtype=dt, device="cuda")
    if op == "append":
        s["pos"] = None  # one axis: the tokens' places in their sequences
        if case["axes"] > 1:
            s["pos"] = torch.randint(0, case["max_ctx"], (case["axes"], T + PAD), generator=g, **i32)
        return s
    s["lse"] = torch.zeros(T + PAD, H, dtype=torch.float32, device="cuda")
    s["tree"] = _trees(case, lens, seed) if case["mask"] == "tree" else None
    return s


# ------------------------------------------------------------------------------ plain forms

def _sin_cos(pos, s):
    """[tokens, 1, rot / 2] each; pos [axes, tokens]; angles in 64 bits."""
    angle = pos.double()[s["axis"].long()].T * s["freqs"][None, :]
    return angle.sin().float()[:, None], angle.cos().float()[:, None]


def _plain_turn(x, sin, cos, case):
    """x [tokens, heads, d] float32 with the first rot elements of every head turned."""
    rot, half = case["rot"], case["rot"] // 2
    y = x.clone()
    if case["style"] == "half":
        a, b = x[..., :half], x[..., half:rot]
        y[..., :half], y[..., half:rot] = a * cos - b * sin, b * cos + a * sin
    else:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        y[..., 0:rot:2], y[..., 1:rot:2] = a * cos - b * sin, b * cos + a * sin
    return y


def _plain_norm(x, weight, s):
    """x over the root of its mean square, times the weight; x float32."""
    if not s["norm"]:
        return x
    return x * torch.rsqrt(x.square().mean(-1, keepdim=True) + s["eps"]) * weight.float()


def _plain_norm_rope(s):
    sin, cos = _sin_cos(s["pos"], s)
    for x in ("q", "k"):
        y = _plain_turn(_plain_norm(s[x].float(), s[x + "_weight"], s), sin, cos, s["case"])
        s[x + "_out"].copy_(y)
    return s["q_out"], s["k_out"]


def _plain_norm_rope_grad(s):
    sin, cos = _sin_cos(s["pos"], s)
    for x in ("q", "k"):
        g = _plain_turn(s["d" + x + "_out"].float(), -sin, cos, s["case"])
        if s["norm"]:
            v, w = s[x].float(), s[x + "_weight"].float()
            r = torch.rsqrt(v.square().mean(-1, keepdim=True) + s["eps"])
            s["d" + x + "_weight"].copy_((g * v * r).sum((0, 1), dtype=torch.float64))
            g = g * w
            g = g * r - v * (r * r * r) * (g * v).mean(-1, keepdim=True)
        s["d" + x].copy_(g)
    out = [s["dqkv"]]
    return out + [s["dq_weight"], s["dk_weight"]] if s["norm"] else out


def _plain_quantise(x):
    """x [..., d] float32 as (float8_e4m3fn values, float8_e8m0fnu powers of two): the smallest
    power that brings the row's largest value within 448."""
    m, e = torch.frexp(x.abs().amax(-1))  # m in [1/2, 1), 448 = 0.875 * 2^9
    e = torch.where(m > 0.875, e - 8, e - 9).clamp(-127, 127)
    up = ((127 - e).clamp(1, 254).to(torch.int32) << 23).view(torch.float32)  # 2^-e
    return (x * up[..., None]).to(torch.float8_e4m3fn), (e + 127).to(torch.uint8).view(
        torch.float8_e8m0fnu)


def _owner(cu, T):
    """(sequence, index in it) of the first T tokens."""
    t = torch.arange(T, device=cu.device)
    b = torch.searchsorted(cu[1:].contiguous(), t.to(torch.int32), right=True)
    return b, t - cu[b]


def _slots(s, T):
    """(page, offset) of the first T tokens' slots, and their places."""
    b, i = _owner(s["cu"], T)
    at = s["before"][b] + i
    return s["table"][b, at // s["case"]["page"]].long(), (at % s["case"]["page"]).long(), at


def _plain_append(s):
    T = s["q"].shape[0] - PAD
    page, slot, at = _slots(s, T)
    sin, cos = _sin_cos(at[None] if s["pos"] is None else s["pos"][:, :T], s)
    q = _plain_norm(s["q"][:T].float(), s["q_weight"], s)
    k = _plain_norm(s["k"][:T].float(), s["k_weight"], s)
    s["o"][:T] = _plain_turn(q, sin, cos, s["case"]).to(s["o"].dtype)
    rows = (("k", _plain_turn(k, sin, cos, s["case"])), ("v", s["v"][:T].float()))
    for x, r in rows:
        y, e = _plain_quantise(r)
        s[x + "_pages"].view(torch.uint8)[page, :, slot] = y.view(torch.uint8)
        s[x + "_scales"].view(torch.uint8)[page, :, slot] = e.view(torch.uint8)
    return [s["o"]] + [s[x] for x in ("k_pages", "v_pages", "k_scales", "v_scales")]


def _values(pages, scales, at):
    """The float32 values of pages[at]."""
    if scales is None:
        return pages[at].float()
    x = pages.view(torch.uint8)[at].view(torch.float8_e4m3fn).float()
    e = scales.view(torch.uint8)[at].to(torch.int32)
    return x * (e.clamp(min=1) << 23).view(torch.float32)[..., None]


def _plain_read(s):
    T = s["k_rows"].shape[0] - PAD
    page, slot, _ = _slots(s, T)
    for x in ("k", "v"):
        at = (page[:, None], torch.arange(s["Hkv"], device="cuda")[None], slot[:, None])
        s[x + "_rows"][:T] = _values(s[x + "_pages"], s[x + "_scales"], at).to(s["k_rows"].dtype)
    return s["k_rows"], s["v_rows"]


def _padded(x, cu, L):
    """Rows of every sequence as [B, L, ...] (rows past its end repeat some row)."""
    rows = cu[:-1, None] + torch.arange(L, device=x.device)[None]
    return x[rows.clamp(max=x.shape[0] - 1)]


def _hidden(s, L, S):
    """[B, 1, 1, L, S]: pairs that the mask or the lengths hide; a chunk's tokens are the last of
    its sequence's keys."""
    case, cu, ctx = s["case"], s["cu"], s["ctx"]
    n = cu[1:] - cu[:-1]
    i = torch.arange(L, device="cuda")[None, :, None]
    j = torch.arange(S, device="cuda")[None, None, :]
    first = (ctx - n)[:, None, None]
    at = i + first
    seen = (i < n[:, None, None]) & (j < ctx[:, None, None])
    if case["mask"] == "tree":
        words = _padded(s["tree"], cu, L).long()  # [B, L, words]
        c = (j - first).expand(len(n), L, S)
        w = words.gather(2, (c // 32).clamp(0, words.shape[2] - 1))
        seen &= (c < 0) | ((w >> (c % 32)) & 1).bool()
    else:
        seen &= j <= at
    if case["mask"] == "window":
        seen &= at - j < case["window"]
    return ~seen[:, None, None]


def _plain_cache(s):
    cu, L, case, Hkv = s["cu"], s["max_new"], s["case"], s["Hkv"]
    width = -(-s["max_ctx"] // case["page"])
    table = s["table"][:, :width].clamp(min=0).long()
    k, v = (_values(s[x + "_pages"], s[x + "_scales"], table).transpose(1, 2).flatten(2, 3)
            for x in ("k", "v"))
    q = _padded(s["q"], cu, L).float()
    B, d = q.shape[0], q.shape[-1]
    G, S = s["H"] // Hkv, k.shape[2]
    q = q.reshape(B, L, Hkv, G, d).permute(0, 2, 3, 1, 4).reshape(B, Hkv, G * L, d)
    p = (q @ k.transpose(2, 3)).mul_(s["scale"]).reshape(B, Hkv, G, L, S)
    p = p.masked_fill_(_hidden(s, L, S), float("-inf"))
    m = p.amax(-1, keepdim=True)
    m = torch.where(m == float("-inf"), torch.zeros_like(m), m)  # a row that sees nothing
    p = p.sub_(m).exp_()
    l = p.sum(-1, keepdim=True)
    o = (p.reshape(B, Hkv, G * L, S) @ v).reshape(B, Hkv, G, L, d) / l.clamp(min=1e-30)
    lse = (m + l.log()).squeeze(-1)
    T = s["q"].shape[0] - PAD
    b, i = _owner(cu, T)
    s["o"][:T] = o.flatten(1, 2)[b, :, i].to(s["o"].dtype)
    s["lse"][:T] = lse.flatten(1, 2)[b, :, i]
    return s["o"], s["lse"]


# ------------------------------------------------------------------------------ one pass

def _workspace(s, size):
    """The workspace that a program keeps beside its buffers."""
    if "workspace" not in s:
        s["workspace"] = torch.empty(max(size(), 16), dtype=torch.uint8, device="cuda")
    return s["workspace"]


def _own_rope(s, fa):
    """The arguments of the calls with a norm and a rotation."""
    case = s["case"]
    kw = dict(style=fa.FA_ROPE_HALF if case["style"] == "half" else fa.FA_ROPE_PAIRS,
              pair_axis=s["axis"] if case["axes"] > 1 else None)
    if s["norm"]:
        kw.update(norm=fa.FA_NORM_RMS, eps=s["eps"], q_weight=s["q_weight"],
                  k_weight=s["k_weight"])
    return kw


def _own_run(s):
    import tiled_attention_06_gb300 as fa
    case, op = s["case"], s["case"]["op"]
    if op == "norm":
        fa.fa_norm_rope(s["q"], s["k"], s["q_out"], s["k_out"], s["pos"], s["freqs"],
                        **_own_rope(s, fa))
        return s["q_out"], s["k_out"]
    if op == "grad":
        kw = _own_rope(s, fa)
        if s["norm"]:
            kw.update(dq_weight=s["dq_weight"], dk_weight=s["dk_weight"],
                      workspace=_workspace(s, lambda: fa.fa_norm_rope_bwd_workspace_size(
                          s["H"], s["Hkv"], case["d"])))
        fa.fa_norm_rope_bwd(s["q"], s["k"], s["dq_out"], s["dk_out"], s["dq"], s["dk"], s["pos"],
                            s["freqs"], **kw)
        return [s["dqkv"]] + ([s["dq_weight"], s["dk_weight"]] if s["norm"] else [])
    if op == "append":
        fa.fa_norm_rope_append(s["q"], s["k"], s["v"], s["o"], s["k_pages"], s["v_pages"],
                               s["table"], s["before"], s["cu"], s["freqs"],
                               k_scales=s["k_scales"], v_scales=s["v_scales"], positions=s["pos"],
                               **_own_rope(s, fa))
        return [s["o"]] + [s[x] for x in ("k_pages", "v_pages", "k_scales", "v_scales")]
    if op == "read":
        fa.fa_kv_read(s["k_pages"], s["v_pages"], s["k_scales"], s["v_scales"], s["table"],
                      s["before"], s["cu"], s["k_rows"], s["v_rows"])
        return s["k_rows"], s["v_rows"]
    ws = _workspace(s, lambda: fa.fa_paged_varlen_workspace_size(
        case["B"], s["H"], s["Hkv"], s["q"].shape[0], s["max_new"], s["table"].shape[1],
        case["page"], case["d"]))
    masks = {"causal": dict(mask_mode=fa.FA_MASK_CAUSAL), "tree": dict(tree=s["tree"]),
             "window": dict(mask_mode=fa.FA_MASK_CAUSAL_WINDOW, window=case["window"])}
    fa.fa_fwd_paged_varlen_ex(s["q"], s["k_pages"], s["v_pages"], s["table"], s["ctx"], s["cu"],
                              s["max_new"], s["o"], s["lse"], s["scale"], ws,
                              k_scales=s["k_scales"], v_scales=s["v_scales"],
                              **masks[case["mask"]])
    return s["o"], s["lse"]


def run(state):
    if own:
        return _own_run(state)
    return {"norm": _plain_norm_rope, "grad": _plain_norm_rope_grad, "append": _plain_append,
            "read": _plain_read, "cache": _plain_cache}[state["case"]["op"]](state)


# ------------------------------------------------------------------------------ in 64 bits

def _turned(x, pos, s, back=False):
    """x [tokens, heads, d] rotated as complex numbers; pos [axes, tokens]."""
    case, rot = s["case"], s["case"]["rot"]
    head, tail = x[..., :rot], x[..., rot:]
    if case["style"] == "half":
        z = torch.complex(head[..., :rot // 2].contiguous(), head[..., rot // 2:].contiguous())
    else:
        z = torch.view_as_complex(head.reshape(*head.shape[:-1], rot // 2, 2).contiguous())
    phase = torch.stack([pos[a].double() * w for a, w in zip(s["axis"].tolist(), s["freqs"])], 1)
    z = z * torch.polar(torch.ones_like(phase), -phase if back else phase)[:, None]
    if case["style"] == "half":
        head = torch.cat([z.real, z.imag], -1)
    else:
        head = torch.view_as_real(z).flatten(-2)
    return torch.cat([head, tail], -1)


def _normed(x, weight, s):
    x = x.double()
    if not s["norm"]:
        return x
    return x / (x.pow(2).sum(-1, keepdim=True) / x.shape[-1] + s["eps"]).sqrt() * weight.double()


def _exact_grad(s):
    """By the chain rule through x = length * direction instead of the collected formula."""
    out, weights = s["dqkv"].double(), []
    for x, at in (("q", slice(0, s["H"])), ("k", slice(s["H"], s["H"] + s["Hkv"]))):
        up = _turned(s["d" + x + "_out"].double(), s["pos"], s, back=True)
        if s["norm"]:
            v = s[x].double()
            rms = (v.pow(2).sum(-1, keepdim=True) / v.shape[-1] + s["eps"]).sqrt()
            n = v / rms
            weights.append((up * n).sum((0, 1)))
            up = up * s[x + "_weight"].double()
            d_rms = -(up * n).sum(-1, keepdim=True) / rms
            up = up / rms + d_rms * v / (v.shape[-1] * rms)
        out[:, at] = up
    return [out] + weights


def _exact_append(s):
    T = s["q"].shape[0] - PAD
    page, slot, at = _slots(s, T)
    pos = at[None] if s["pos"] is None else s["pos"][:, :T]
    o = s["o"].double()
    o[:T] = _turned(_normed(s["q"][:T], s["q_weight"], s), pos, s)
    rows = dict(k=_turned(_normed(s["k"][:T], s["k_weight"], s), pos, s), v=s["v"][:T].double())
    out = {}
    for x, r in rows.items():
        # a largest value of 448 times a power of two itself needs no more than that power
        power = torch.pow(2.0, torch.ceil(torch.log2(r.abs().amax(-1) / 448) - 1e-12))
        out[x + "_pages"], out[x + "_scales"] = s[x + "_pages"].double(), s[x + "_scales"].double()
        out[x + "_pages"][page, :, slot] = r / power[..., None]  # before the rounding to 8 bits
        out[x + "_scales"][page, :, slot] = power
    return [o] + [out[x] for x in ("k_pages", "v_pages", "k_scales", "v_scales")]


def _rows_of(s, x, b, first, last):
    """[Hkv, last - first, d] of sequence b in 64 bits."""
    pages = s["table"][b, first // s["case"]["page"]:-(-last // s["case"]["page"])].long()
    skip = first % s["case"]["page"]
    y = s[x + "_pages"].view(torch.uint8)[pages].view(s[x + "_pages"].dtype).double()
    if s[x + "_scales"] is not None:
        e = s[x + "_scales"].view(torch.uint8)[pages].double() - 127
        y = y * torch.pow(2.0, e)[..., None]
    return y.transpose(0, 1).flatten(1, 2)[:, skip:skip + last - first]


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "norm":
        return tuple(_turned(_normed(s[x], s[x + "_weight"], s), s["pos"], s) for x in ("q", "k"))
    if case["op"] == "grad":
        return _exact_grad(s)
    if case["op"] == "append":
        return _exact_append(s)
    at = 0
    if case["op"] == "read":
        out = [s["k_rows"].double(), s["v_rows"].double()]
        for b, (n, c) in enumerate(_lengths(case)):
            for x, y in zip("kv", out):
                y[at:at + n] = _rows_of(s, x, b, c, c + n).transpose(0, 1)
            at += n
        return tuple(out)
    o, lse, G = s["o"].double(), s["lse"].double(), s["H"] // s["Hkv"]
    for b, (n, c) in enumerate(_lengths(case)):
        k, v = (_rows_of(s, x, b, 0, n + c) for x in "kv")
        i, j = torch.arange(c, c + n, device="cuda")[:, None], torch.arange(n + c, device="cuda")[None]
        seen = j <= i
        if case["mask"] == "window":
            seen = seen & (j > i - case["window"])
        if case["mask"] == "tree":
            mine = torch.arange(n, device="cuda")
            bits = s["tree"][at:at + n].long()[:, mine // 32] >> (mine % 32) & 1
            seen = torch.cat([torch.ones(n, c, dtype=torch.bool, device="cuda"), bits.bool()], 1)
        bias = torch.zeros(n, n + c, dtype=torch.float64, device="cuda").masked_fill(
            ~seen, float("-inf"))
        for h in range(s["H"]):
            x = s["q"][at:at + n, h].double() @ k[h // G].T * s["scale"] + bias
            lse[at:at + n, h] = torch.logsumexp(x, -1)
            o[at:at + n, h] = torch.softmax(x, -1) @ v[h // G]
        at += n
    return o, lse
