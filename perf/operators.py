"""Rotary positions, attention over packed prompts with grouped heads (and its gradient), and
attention of new tokens over a paged cache: the cases they are measured on, their plain form in
elementary torch operations, and the framework's calls.

Layouts: tokens are packed, [tokens, heads, d]; sequence b owns the rows cu[b] .. cu[b+1]-1.
Pools are [num_pages, kv_heads, page, d] with an int32 block table per sequence. Query head h
reads K/V head h // (H // Hkv).
"""
import math
import random

import torch

own = False

DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
MAX_SCORES = 8 * 32 * 4096 * 4096  # padded scores of the largest listed case


# ------------------------------------------------------------------------------ cases

def listed():
    return [
        # one step of 64 sequences far into long contexts: the q and k heads of the fused
        # projection, one token each
        dict(name="rope_step", op="rope", T=64, H=32, Hkv=8, d=128, rot=128, style="half",
             scaling="plain", inverse=False, dtype="bf16", max_pos=1 << 20),
        # the prompts of a batch, whole heads
        dict(name="rope_prompt", op="rope", T=16384, H=32, Hkv=8, d=128, rot=128, style="half",
             scaling="plain", inverse=False, dtype="bf16", max_pos=8192),
        # the gradient of an interleaved rotation of half the head, scaled for long contexts,
        # odd number of tokens
        dict(name="rope_grad", op="rope", T=8191, H=16, Hkv=4, d=128, rot=64, style="pairs",
             scaling="yarn", inverse=True, dtype="f16", max_pos=65536),
        # one new token for each of 64 sequences into the cache
        dict(name="append_step", op="append", B=64, H=32, Hkv=8, d=128, rot=128, style="half",
             scaling="plain", dtype="bf16", page=256, max_ctx=2048, max_new=1, lens_seed=1),
        # ragged chunks of up to 512 tokens of eight sequences, 64-token pages
        dict(name="append_chunk", op="append", B=8, H=32, Hkv=8, d=128, rot=128, style="half",
             scaling="linear", dtype="f16", page=64, max_ctx=8192, max_new=512, lens_seed=2),
        # sixteen short prompts of a chat batch
        dict(name="packed_short", op="packed", B=16, H=32, Hkv=8, d=128, mask="causal", window=0,
             dtype="bf16", min_len=1, max_len=256, lens_seed=3),
        # eight prompts of up to 4096 tokens
        dict(name="packed_long", op="packed", B=8, H=32, Hkv=8, d=128, mask="causal", window=0,
             dtype="bf16", min_len=512, max_len=4096, lens_seed=4),
        # training on short documents packed into one row, d = 64, three query heads a group
        dict(name="grad_short", op="grad", B=24, H=12, Hkv=4, d=64, mask="causal", window=0,
             dtype="f16", min_len=1, max_len=320, lens_seed=5),
        # training on long documents
        dict(name="grad_long", op="grad", B=4, H=32, Hkv=8, d=128, mask="causal", window=0,
             dtype="bf16", min_len=512, max_len=4096, lens_seed=6),
        # one token per sequence over contexts of up to 8192 tokens
        dict(name="cache_step", op="cache", B=32, H=32, Hkv=8, d=128, mask="causal", window=0,
             dtype="f16", page=256, max_ctx=8192, min_new=1, max_new=1, lens_seed=7),
        # a few drafted tokens checked at once over long contexts, 64-token pages
        dict(name="cache_draft", op="cache", B=4, H=32, Hkv=4, d=128, mask="causal", window=0,
             dtype="bf16", page=64, max_ctx=65536, min_new=5, max_new=5, lens_seed=8),
        # chunks of a prompt next to what is cached of it
        dict(name="cache_chunk", op="cache", B=8, H=32, Hkv=8, d=128, mask="causal", window=0,
             dtype="bf16", page=256, max_ctx=8192, min_new=1, max_new=512, lens_seed=9),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["rope", "append", "packed", "grad", "cache"])
    hkv = rng.choice([1, 2, 3, 4, 8])
    heads = dict(H=hkv * rng.choice([1, 2, 3, 4, 5, 7, 8]), Hkv=hkv)
    d = rng.choice([64, 128])
    if op in ("rope", "append"):
        rope = dict(rot=d if rng.random() < 0.5 else 2 * rng.randint(1, d // 2),
                    style=rng.choice(["half", "pairs"]),
                    scaling=rng.choice(["plain", "linear", "yarn"]))
    if op == "rope":
        heads = dict(H=min(heads["H"], 32), Hkv=hkv)
        return dict(op=op, T=_log(rng, 1, 16384), d=d, inverse=rng.random() < 0.5,
                    dtype=rng.choice(["f16", "bf16", "bf16", "f32"]) if d == 64 else
                    rng.choice(["f16", "bf16"]),
                    max_pos=_log(rng, 16, 1 << 20), **heads, **rope)
    seed = rng.randrange(1 << 30)
    dtype = rng.choice(["f16", "bf16"])
    page = rng.choice([16, 64, 128, 256])
    if op == "append":
        return dict(op=op, B=_log(rng, 1, 64), d=d, dtype=dtype, page=page,
                    max_ctx=_log(rng, 600, 2048), max_new=_log(rng, 1, 256), lens_seed=seed,
                    **heads, **rope)
    mask = rng.choice(["causal", "causal", "causal", "window"])
    window = _log(rng, 1, 2048) if mask == "window" else 0
    if op in ("packed", "grad"):
        B, hi = _log(rng, 1, 64), _log(rng, 1, 4096)
        most = MAX_SCORES // (1 if op == "packed" else 2)
        while B * heads["H"] * hi * hi > most:
            B, hi = max(1, B * 3 // 4), max(1, hi * 4 // 5)
        return dict(op=op, B=B, d=d, mask=mask, window=window, dtype=dtype, min_len=1,
                    max_len=hi, lens_seed=seed, **heads)
    B, ctx, new = _log(rng, 1, 64), _log(rng, 64, 32768), rng.choice([1, 1, _log(rng, 1, 512)])
    while B * ctx * hkv > 32 * 8192 * 8 or B * heads["H"] * new * ctx > MAX_SCORES // 16:
        B, ctx, new = max(1, B * 3 // 4), max(64, ctx * 7 // 8), max(1, new * 7 // 8)
    return dict(op=op, B=B, d=d, mask=mask, window=window, dtype=dtype, page=page, max_ctx=ctx,
                min_new=1, max_new=min(new, ctx), lens_seed=seed, **heads)


def _lengths(case):
    """(tokens, tokens cached before them) of every sequence."""
    rng = random.Random(case["lens_seed"])
    if case["op"] in ("packed", "grad"):
        return [(rng.randint(case["min_len"], case["max_len"]), 0) for _ in range(case["B"])]
    out = []
    for _ in range(case["B"]):
        n = rng.randint(case.get("min_new", 1), case["max_new"])
        total = rng.randint(n, max(n, case["max_ctx"]))
        out.append((n, total - n))
    return out


def _visible_pairs(case, n, before):
    """Visible (query, key) pairs of one sequence and head."""
    w = case["window"] if case["mask"] == "window" else n + before
    full = max(0, min(n, w - before))  # queries that see every earlier key
    return full * before + full * (full + 1) // 2 + (n - full) * w


def work(case):
    d, H, Hkv = case["d"], case["H"], case["Hkv"]
    e = 4 if case["dtype"] == "f32" else 2
    if case["op"] == "rope":
        n = case["T"] * (H + Hkv)
        return {"bytes": 2 * n * d * e + case["T"] * 4 + case["rot"] // 2 * 8,
                "flops": n * case["rot"] * 3}
    lens = _lengths(case)
    T = sum(n for n, _ in lens)
    if case["op"] == "append":
        return {"bytes": T * (H + 2 * Hkv) * d * e * 2, "flops": T * (H + Hkv) * case["rot"] * 3}
    pairs = sum(_visible_pairs(case, n, c) for n, c in lens) * H
    if case["op"] == "packed":
        return {"bytes": T * (2 * H + 2 * Hkv) * d * e + T * H * 4, "flops": 4 * d * pairs}
    if case["op"] == "grad":
        return {"bytes": T * (4 * H + 4 * Hkv) * d * e + T * H * 4, "flops": 10 * d * pairs}
    keys = sum(min(n + c, case["window"] + n - 1) if case["mask"] == "window" else n + c
               for n, c in lens)
    return {"bytes": keys * 2 * Hkv * d * e + T * 2 * H * d * e + T * H * 4,
            "flops": 4 * d * pairs}


# ------------------------------------------------------------------------------ inputs

def _frequencies(case):
    """Radians per position of every rotated pair (float64), and the amplitude."""
    rot, base = case["rot"], 10000.0
    i = torch.arange(rot // 2, dtype=torch.float64, device="cuda")
    w = base ** (-2.0 * i / rot)
    if case["scaling"] == "plain":
        return w, 1.0
    if case["scaling"] == "linear":
        return w / 4.0, 1.0
    factor, trained = 8.0, 4096.0  # low frequencies divided by the factor, high ones kept
    turns = trained * w / (2 * math.pi)
    keep = ((turns - 1.0) / (32.0 - 1.0)).clamp(0.0, 1.0)
    return w * keep + w / factor * (1 - keep), 0.1 * math.log(factor) + 1.0


def _pages(case, lens, g):
    """Block table over a pool whose pages are taken in random order, and the pool's size."""
    need = [-(-(n + c) // case["page"]) for n, c in lens]
    pool = sum(need) + 3
    order = torch.randperm(pool, generator=torch.Generator().manual_seed(int(g) + 7)).tolist()
    width = max(need) + 1
    table = [[-1] * width for _ in lens]
    at = 0
    for b, k in enumerate(need):
        table[b][:k] = order[at:at + k]
        at += k
    return torch.tensor(table, dtype=torch.int32, device="cuda"), pool


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    dt, d, H, Hkv = DTYPES[case["dtype"]], case["d"], case["H"], case["Hkv"]

    def randn(*shape):
        return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32).to(dt)

    s = {"case": case, "H": H, "Hkv": Hkv, "scale": 1.0 / math.sqrt(d)}
    if case["op"] in ("rope", "append"):
        s["freqs"], s["amplitude"] = _frequencies(case)
    if case["op"] == "rope":
        T = case["T"]
        qkv = randn(T, H + 2 * Hkv, d)  # the fused projection; v is not rotated
        s["x"] = qkv[:, :H + Hkv]
        s["pos"] = torch.randint(0, case["max_pos"], (T,), generator=g, device="cuda",
                                 dtype=torch.int32)
        s["y"] = torch.zeros(T, H + Hkv, d, dtype=dt, device="cuda")
        return s
    lens = _lengths(case)
    new, before = [n for n, _ in lens], [c for _, c in lens]
    T, pad = sum(new), 3  # three rows behind the last sequence belong to nobody
    i32 = dict(dtype=torch.int32, device="cuda")
    s["cu"] = torch.tensor([sum(new[:b]) for b in range(len(new) + 1)], **i32)
    s["max_new"], s["max_ctx"] = max(new), max(n + c for n, c in lens)
    qkv = randn(T + pad, H + 2 * Hkv, d)
    s["q"], s["k"], s["v"] = qkv[:, :H], qkv[:, H:H + Hkv], qkv[:, H + Hkv:]
    s["o"] = torch.zeros(T + pad, H, d, dtype=dt, device="cuda")
    if case["op"] in ("append", "cache"):
        s["table"], pool = _pages(case, lens, seed)
        s["k_pages"], s["v_pages"] = (randn(pool, Hkv, case["page"], d) for _ in range(2))
        s["before"] = torch.tensor(before, **i32)
        s["ctx"] = torch.tensor([n + c for n, c in lens], **i32)
    if case["op"] != "append":
        s["lse"] = torch.zeros(T + pad, H, dtype=torch.float32, device="cuda")
    if case["op"] == "grad":
        _plain_packed(s)  # the forward's outputs, which a training step has kept
        s["dout"] = randn(T + pad, H, d)
        s["dq"] = torch.zeros(T + pad, H, d, dtype=dt, device="cuda")
        s["dk"], s["dv"] = (torch.zeros(T + pad, Hkv, d, dtype=dt, device="cuda")
                            for _ in range(2))
    return s


# ------------------------------------------------------------------------------ plain forms

def _plain_rotate(x, pos, s):
    """x [tokens, heads, d] float32, rotated; angles in 64 bits."""
    case = s["case"]
    rot, half = case["rot"], case["rot"] // 2
    angle = pos.double()[:, None] * s["freqs"][None, :]
    if case.get("inverse"):
        angle = -angle
    cos = (angle.cos() * s["amplitude"]).float()[:, None]
    sin = (angle.sin() * s["amplitude"]).float()[:, None]
    y = x.clone()
    if case["style"] == "half":
        a, b = x[..., :half], x[..., half:rot]
        y[..., :half], y[..., half:rot] = a * cos - b * sin, b * cos + a * sin
    else:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        y[..., 0:rot:2], y[..., 1:rot:2] = a * cos - b * sin, b * cos + a * sin
    return y


def _owner(cu, T):
    """(sequence, index in it) of the first T tokens."""
    t = torch.arange(T, device=cu.device)
    b = torch.searchsorted(cu[1:].contiguous(), t.to(torch.int32), right=True)
    return b, t - cu[b]


def _plain_append(s):
    case, cu = s["case"], s["cu"]
    T = s["q"].shape[0] - 3
    b, i = _owner(cu, T)
    pos = s["before"][b] + i
    q = _plain_rotate(s["q"][:T].float(), pos, s)
    k = _plain_rotate(s["k"][:T].float(), pos, s)
    s["o"][:T] = q.to(s["o"].dtype)
    page = s["table"][b, pos // case["page"]].long()
    slot = (pos % case["page"]).long()
    s["k_pages"][page, :, slot] = k.to(s["o"].dtype)
    s["v_pages"][page, :, slot] = s["v"][:T]
    return s["o"], s["k_pages"], s["v_pages"]


def _padded(x, cu, L):
    """Rows of every sequence as [B, L, ...] float32 (rows past its end repeat some row)."""
    rows = cu[:-1, None] + torch.arange(L, device=x.device)[None]
    return x[rows.clamp(max=x.shape[0] - 1)].float()


def _hidden(case, n, total, L, S, device):
    """[B, 1, 1, L, S]: pairs that the mask or the lengths hide; n queries are the last of
    `total` keys."""
    i = torch.arange(L, device=device)[None, :, None]
    j = torch.arange(S, device=device)[None, None, :]
    at = i + (total - n)[:, None, None]
    seen = (i < n[:, None, None]) & (j <= at) & (j < total[:, None, None])
    if case["mask"] == "window":
        seen &= at - j < case["window"]
    return ~seen[:, None, None]


def _scores(q, k, hidden, scale):
    """[B, Hkv, G, L, S] scaled scores, -inf where hidden; q [B, L, H, d], k [B, Hkv, S, d]."""
    B, L, H, d = q.shape
    Hkv = k.shape[1]
    qg = q.reshape(B, L, Hkv, H // Hkv, d).permute(0, 2, 3, 1, 4).reshape(B, Hkv, -1, d)
    s = (qg @ k.transpose(2, 3)).mul_(scale).reshape(B, Hkv, H // Hkv, L, -1)
    return s.masked_fill_(hidden, float("-inf"))


def _softmax_v(s, v):
    """Softmax over the last axis times v, and the log of the sum; a row that sees nothing
    gives 0 and -inf."""
    m = s.amax(-1, keepdim=True)
    m = torch.where(m == float("-inf"), torch.zeros_like(m), m)
    p = s.sub_(m).exp_()
    l = p.sum(-1, keepdim=True)
    B, Hkv, G, L, S = p.shape
    o = (p.reshape(B, Hkv, G * L, S) @ v).reshape(B, Hkv, G, L, -1)
    return o / l.clamp(min=1e-30), (m + l.log()).squeeze(-1)


def _put_rows(s, o, lse, T):
    """[B, Hkv, G, L, d] and [B, Hkv, G, L] into the packed rows."""
    b, i = _owner(s["cu"], T)
    s["o"][:T] = o.flatten(1, 2)[b, :, i].to(s["o"].dtype)
    s["lse"][:T] = lse.flatten(1, 2)[b, :, i]
    return s["o"], s["lse"]


def _plain_packed(s):
    cu, L = s["cu"], s["max_new"]
    n = cu[1:] - cu[:-1]
    q, k, v = (_padded(s[x], cu, L) for x in ("q", "k", "v"))
    hidden = _hidden(s["case"], n, n, L, L, q.device)
    o, lse = _softmax_v(_scores(q, k.transpose(1, 2), hidden, s["scale"]), v.transpose(1, 2))
    return _put_rows(s, o, lse, s["q"].shape[0] - 3)


def _plain_grad(s):
    cu, L, H, Hkv = s["cu"], s["max_new"], s["H"], s["Hkv"]
    T, G = s["q"].shape[0] - 3, H // Hkv
    n = cu[1:] - cu[:-1]
    q, k, v, o, do, lse = (_padded(s[x], cu, L) for x in ("q", "k", "v", "o", "dout", "lse"))
    B, d = q.shape[0], q.shape[-1]

    def grouped(x):  # [B, L, H, ...] -> [B, Hkv, G * L, ...]
        x = x.reshape(B, L, Hkv, G, -1).permute(0, 2, 3, 1, 4)
        return x.reshape(B, Hkv, G * L, -1)

    kt, vt = k.transpose(1, 2), v.transpose(1, 2)
    hidden = _hidden(s["case"], n, n, L, L, q.device)
    p = _scores(q, kt, hidden, s["scale"]).reshape(B, Hkv, G * L, L)
    p = p.sub_(grouped(lse[..., None])).exp_()
    seen = ~hidden.expand(B, 1, G, L, L).reshape(B, 1, G * L, L)
    p = torch.where(seen, p, torch.zeros((), device=p.device))
    # rows past a sequence's end are hidden, but their dout belongs to another sequence
    live = (torch.arange(L, device=q.device)[None] < n[:, None])[:, :, None, None]
    do, o, q = do * live, o * live, q * live
    dog, qg = grouped(do), grouped(q)
    dv = p.transpose(2, 3) @ dog
    dp = dog @ vt.transpose(2, 3)
    ds = dp.sub_(grouped((do * o).sum(-1, keepdim=True))).mul_(p).mul_(s["scale"])
    dq = (ds @ kt).reshape(B, H, L, d)
    dk = ds.transpose(2, 3) @ qg
    b, i = _owner(cu, T)
    for name, x in (("dq", dq), ("dk", dk), ("dv", dv)):
        s[name][:T] = x[b, :, i].to(s[name].dtype)
    return s["dq"], s["dk"], s["dv"]


def _plain_cache(s):
    cu, L, ctx, case = s["cu"], s["max_new"], s["ctx"], s["case"]
    n = cu[1:] - cu[:-1]
    width = -(-s["max_ctx"] // case["page"])
    table = s["table"][:, :width].clamp(min=0).long()
    k, v = (x[table].transpose(1, 2).flatten(2, 3).float() for x in (s["k_pages"], s["v_pages"]))
    hidden = _hidden(case, n, ctx, L, k.shape[2], k.device)
    o, lse = _softmax_v(_scores(_padded(s["q"], cu, L), k, hidden, s["scale"]), v)
    return _put_rows(s, o, lse, s["q"].shape[0] - 3)


# ------------------------------------------------------------------------------ one pass

def _own_masks(fa, case):
    if case["mask"] == "window":
        return dict(mask_mode=fa.FA_MASK_CAUSAL_WINDOW, window=case["window"])
    return dict(mask_mode=fa.FA_MASK_CAUSAL)


def _workspace(s, size):
    """The workspace that a program keeps beside its buffers."""
    if "workspace" not in s:
        s["workspace"] = torch.empty(max(size(), 16), dtype=torch.uint8, device="cuda")
    return s["workspace"]


def _own_run(s):
    import tiled_attention_06_gb300 as fa
    case, op = s["case"], s["case"]["op"]
    if op in ("rope", "append"):
        style = fa.FA_ROPE_HALF if case["style"] == "half" else fa.FA_ROPE_PAIRS
    if op == "rope":
        fa.fa_rope(s["x"], s["y"], s["pos"], s["freqs"], style, s["amplitude"], case["inverse"])
        return s["y"]
    if op == "append":
        fa.fa_rope_append(s["q"], s["k"], s["v"], s["o"], s["k_pages"], s["v_pages"], s["table"],
                          s["before"], s["cu"], s["freqs"], style, s["amplitude"])
        return s["o"], s["k_pages"], s["v_pages"]
    B, T, d = case["B"], s["q"].shape[0], case["d"]
    if op == "packed":
        ws = _workspace(s, lambda: fa.fa_varlen_workspace_size(B, s["H"], s["Hkv"], T, T, d))
        fa.fa_fwd_varlen(s["q"], s["k"], s["v"], s["o"], s["lse"], s["cu"], s["cu"], s["scale"],
                         ws, **_own_masks(fa, case))
        return s["o"], s["lse"]
    if op == "grad":
        ws = _workspace(s, lambda: fa.fa_bwd_varlen_workspace_size(B, s["H"], s["Hkv"], T, T, d))
        fa.fa_bwd_varlen(s["q"], s["k"], s["v"], s["o"], s["dout"], s["lse"], s["dq"], s["dk"],
                         s["dv"], s["cu"], s["cu"], s["scale"], ws, **_own_masks(fa, case))
        return s["dq"], s["dk"], s["dv"]
    ws = _workspace(s, lambda: fa.fa_paged_varlen_workspace_size(
        B, s["H"], s["Hkv"], T, s["max_new"], s["table"].shape[1], case["page"], d))
    fa.fa_fwd_paged_varlen(s["q"], s["k_pages"], s["v_pages"], s["table"], s["ctx"], s["cu"],
                           s["max_new"], s["o"], s["lse"], s["scale"], ws,
                           **_own_masks(fa, case))
    return s["o"], s["lse"]


def run(state):
    if own:
        return _own_run(state)
    op = state["case"]["op"]
    if op == "rope":
        state["y"].copy_(_plain_rotate(state["x"].float(), state["pos"], state))
        return state["y"]
    return {"append": _plain_append, "packed": _plain_packed, "grad": _plain_grad,
            "cache": _plain_cache}[op](state)


# ------------------------------------------------------------------------------ in 64 bits

def _turned(x, pos, s):
    """x [tokens, heads, d] rotated as complex numbers in 64 bits."""
    case, rot = s["case"], s["case"]["rot"]
    x = x.double()
    head, tail = x[..., :rot], x[..., rot:]
    if case["style"] == "half":
        z = torch.complex(head[..., :rot // 2].contiguous(), head[..., rot // 2:].contiguous())
    else:
        z = torch.view_as_complex(head.reshape(*head.shape[:-1], rot // 2, 2).contiguous())
    phase = torch.outer(pos.double(), s["freqs"]) * (-1.0 if case.get("inverse") else 1.0)
    z = z * torch.polar(torch.full_like(phase, s["amplitude"]), phase)[:, None]
    if case["style"] == "half":
        head = torch.cat([z.real, z.imag], -1)
    else:
        head = torch.view_as_real(z).flatten(-2)
    return torch.cat([head, tail], -1)


def _bias(case, n, total):
    at = torch.arange(total - n, total, device="cuda")[:, None]
    j = torch.arange(total, device="cuda")[None]
    seen = j <= at
    if case["mask"] == "window":
        seen = seen & (j > at - case["window"])
    return torch.zeros(n, total, dtype=torch.float64, device="cuda").masked_fill(
        ~seen, float("-inf"))


def _exact_head(q, k, v, bias, scale):
    s = q.double() @ k.double().T * scale + bias
    lse = torch.logsumexp(s, -1)
    return torch.exp(s - lse[:, None]), lse


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "rope":
        return _turned(s["x"], s["pos"], s)
    lens, at = _lengths(case), 0
    o = s["o"].double()
    if case["op"] == "append":
        kp, vp = s["k_pages"].double(), s["v_pages"].double()
        for b, (n, c) in enumerate(lens):
            pos = torch.arange(c, c + n, device="cuda")
            o[at:at + n] = _turned(s["q"][at:at + n], pos, s)
            page, slot = s["table"][b].long()[pos // case["page"]], pos % case["page"]
            kp[page, :, slot] = _turned(s["k"][at:at + n], pos, s)
            vp[page, :, slot] = s["v"][at:at + n].double()
            at += n
        return o, kp, vp
    G = s["H"] // s["Hkv"]
    lse = s["lse"].double()
    grads = [s[x].double() for x in ("dq", "dk", "dv")] if case["op"] == "grad" else None
    for b, (n, c) in enumerate(lens):
        rows = slice(at, at + n)
        bias = _bias(case, n, n + c)
        for h in range(s["H"]):
            if case["op"] == "cache":
                pages = s["table"][b, :-(-(n + c) // case["page"])].long()
                k, v = (x[pages, h // G].flatten(0, 1)[:n + c]
                        for x in (s["k_pages"], s["v_pages"]))
            else:
                k, v = s["k"][rows, h // G], s["v"][rows, h // G]
            p, l = _exact_head(s["q"][rows, h], k, v, bias, s["scale"])
            oh = p @ v.double()
            if grads is None:
                o[rows, h], lse[rows, h] = oh, l
                continue
            do = s["dout"][rows, h].double()
            ds = p * (do @ v.double().T - (do * oh).sum(-1, keepdim=True)) * s["scale"]
            grads[0][rows, h] = ds @ k.double()
            grads[1][rows, h // G] += ds.T @ s["q"][rows, h].double()
            grads[2][rows, h // G] += p.T @ do
        at += n
    return tuple(grads) if grads is not None else (o, lse)
