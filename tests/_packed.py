"""Plain implementations in 64 bits for the calls over packed tokens, and their tolerances.

Tolerances. u = eps(dtype) / 2 is the largest relative error of one rounding (bf16 2^-8, fp16
2^-11).

Forward. P is rounded once to 16 bits (each term of the numerator off by at most u of itself), the
row sum is not, and O is rounded once: |O - O_ref| <= u sum_j P_j |v_j| / l + u |O| + small <=
2 u max|v| over the row's visible keys. FP32 exponentials and sums add at most about 2^-18.
LSE: scores are FP32 sums of d exact products (error below d 2^-24 sum |q k| scale) and the
logarithm's and exponentials' approximations stay below 2^-20 absolute each: 1e-4 for the
inputs here (|scores| < 100, d <= 128).

Gradients. P and dS are rounded to 16 bits, o is rounded (which moves D = dout . o), and so are
the results. With |dS|_ij = P_ij (|dP_ij| + |D_i|), to first order in u:
    |dv - ref| <= u (P^T |dout|) + u |dv|
    |dk - ref| <= scale (u (|dS|^T |q|) + u (E^T |q|)) + u |dk|,  E_ij = P_ij (|dout| . |o|)_i
    |dq - ref| <= scale (u |dS| |k| + u E |k|) + u |dq|
where E is what the rounding of o moves dS by. FP32 accumulation and the LSE's own rounding
(P off by 2^-18 of itself) add about 2^-16 of the same sums. gradients() evaluates them.
"""
import torch

import tiled_attention_06_gb300 as fa


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def seen(n, m, mask, window=0, n_global=0):
    """[n, m] bool: does query i (one of the last n of m positions) see key j?"""
    i = torch.arange(n)[:, None] + (m - n)
    j = torch.arange(m)[None]
    if mask == fa.FA_MASK_NONE:
        return torch.ones(n, m, dtype=torch.bool)
    if mask == fa.FA_MASK_CAUSAL:
        return j <= i
    if mask == fa.FA_MASK_CAUSAL_WINDOW:
        return (j <= i) & ((i - j < window) | (j < n_global))
    if mask == fa.FA_MASK_BAND:
        return (i - j).abs() <= window
    return (j <= i) | (j < n_global)


def head(q, k, v, vis, scale):
    """(P, O, LSE) of one sequence and head in 64 bits; empty rows give 0 and -inf."""
    s = q.double() @ k.double().T * scale
    s = s.masked_fill(~vis, float("-inf"))
    if s.shape[1] == 0:
        return s, torch.zeros(q.shape[0], q.shape[1], dtype=torch.float64), \
            torch.full((q.shape[0],), float("-inf"), dtype=torch.float64)
    lse = torch.logsumexp(s, -1)
    p = torch.where(vis, torch.exp(s - torch.where(lse.isinf(), 0.0, lse)[:, None]),
                    torch.zeros((), dtype=torch.float64))
    return p, p @ v.double(), lse


def attention(q, k, v, cu_q, cu_k, scale, mask, window=0, n_global=0):
    """Packed attention, CPU tensors: o, lse and the bound on |o - o_ref| without u."""
    T, H, d = q.shape
    G = H // k.shape[1]
    o = torch.zeros(T, H, d, dtype=torch.float64)
    lse = torch.zeros(T, H, dtype=torch.float64)
    bound = torch.zeros(T, H, dtype=torch.float64)
    for b in range(len(cu_q) - 1):
        rq, rk = slice(cu_q[b], cu_q[b + 1]), slice(cu_k[b], cu_k[b + 1])
        vis = seen(cu_q[b + 1] - cu_q[b], cu_k[b + 1] - cu_k[b], mask, window, n_global)
        for h in range(H):
            p, oh, l = head(q[rq, h], k[rk, h // G], v[rk, h // G], vis, scale)
            o[rq, h], lse[rq, h] = oh, l
            if vis.shape[1]:
                big = v[rk, h // G].double().abs().amax(-1)
                bound[rq, h] = (vis * big[None]).amax(-1)
    return o, lse, bound


def check_forward(o, lse, ref, dtype, rows, what=""):
    """o, lse from the GPU against attention()'s, over the first `rows` packed rows."""
    ro, rl, bound = ref
    u = half_step(dtype)
    got = o[:rows].double().cpu()
    assert torch.isfinite(got).all(), f"{what}: non-finite"
    err = (got - ro[:rows]).abs().amax(-1)
    lim = 2 * u * bound[:rows] + 2.0 ** -18 * (1 + bound[:rows])
    assert (err <= lim).all(), f"{what}: |dO| {float((err - lim).max()):.3e} over its bound"
    if lse is not None:
        gl = lse[:rows].double().cpu()
        inf = rl[:rows].isinf()
        assert torch.equal(gl.isneginf(), inf), f"{what}: -inf pattern"
        if (~inf).any():
            e = float((gl - rl[:rows])[~inf].abs().max())
            assert e <= 1e-4, f"{what}: |dLSE| {e:.3e}"


def starts(lengths):
    out = [0]
    for n in lengths:
        out.append(out[-1] + n)
    return out


def rotate(x, pos, freqs, rot, half, amplitude=1.0, inverse=False):
    """x [T, H, d] rotated in 64 bits."""
    y = x.double().clone()
    t = pos.double()[:, None, None] * freqs.double()[None, None] * (-1 if inverse else 1)
    c, s = t.cos() * amplitude, t.sin() * amplitude
    if half:
        ia, ib = torch.arange(rot // 2), torch.arange(rot // 2, rot)
    else:
        ia, ib = torch.arange(0, rot, 2), torch.arange(1, rot, 2)
    a, b = x.double()[..., ia], x.double()[..., ib]
    y[..., ia] = a * c - b * s
    y[..., ib] = b * c + a * s
    return y


def gradients(q, k, v, dout, cu_q, cu_k, scale, dtype, mask, window=0, n_global=0):
    """[(dq, bound), (dk, bound), (dv, bound)] in 64 bits, CPU tensors."""
    u, slack = half_step(dtype), 2.0 ** -16
    G = q.shape[1] // k.shape[1]
    out = [[torch.zeros(x.shape, dtype=torch.float64) for _ in range(2)] for x in (q, k, v)]
    for b in range(len(cu_q) - 1):
        rq, rk = slice(cu_q[b], cu_q[b + 1]), slice(cu_k[b], cu_k[b + 1])
        vis = seen(cu_q[b + 1] - cu_q[b], cu_k[b + 1] - cu_k[b], mask, window, n_global)
        for h in range(q.shape[1]):
            hk = h // G
            qh, kh, vh, do = (x.double() for x in (q[rq, h], k[rk, hk], v[rk, hk], dout[rq, h]))
            p, o, _ = head(qh, kh, vh, vis, scale)
            if p.shape[1] == 0:
                continue
            dp, dsum = do @ vh.T, (do * o).sum(-1, keepdim=True)
            ds = p * (dp - dsum)
            big = p * (dp.abs() + dsum.abs())
            e = p * (do.abs() * o.abs()).sum(-1, keepdim=True)
            w = (u + slack) * big + u * e
            out[0][0][rq, h] = scale * ds @ kh
            out[0][1][rq, h] = scale * w @ kh.abs()
            out[1][0][rk, hk] += scale * ds.T @ qh
            out[1][1][rk, hk] += scale * w.T @ qh.abs()
            out[2][0][rk, hk] += p.T @ do
            out[2][1][rk, hk] += (u + slack) * (p.T @ do.abs())
    return [(ref, bound + u * (ref.abs() + bound) + 2.0 ** -24) for ref, bound in out]


def check_gradients(got, ref, rows_q, rows_k, what=""):
    for name, x, (r, bound), rows in zip(("dq", "dk", "dv"), got, ref, (rows_q, rows_k, rows_k)):
        x = x[:rows].double().cpu()
        assert torch.isfinite(x).all(), f"{what} {name}: non-finite"
        over = (x - r[:rows]).abs() - bound[:rows]
        assert (over <= 0).all(), f"{what} {name}: {float(over.max()):.3e} over its bound"
