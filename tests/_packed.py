"""Plain implementations in 64 bits for the calls over packed tokens, and their tolerances.

Tolerances. u = eps(dtype) / 2 is the largest relative error of one rounding (bf16 2^-8, fp16
2^-11).

Forward. P is rounded once to 16 bits (each term of the numerator off by at most u of itself), the
row sum is not, and O is rounded once: |O - O_ref| <= u sum_j P_j |v_j| / l + u |O| + small <=
2 u max|v| over the row's visible keys. FP32 exponentials and sums add at most about 2^-18.
LSE: scores are FP32 sums of d exact products (error below d 2^-24 sum |q k| scale) and the
logarithm's and exponentials' approximations stay below 2^-20 absolute each: 1e-4 for the
inputs here (|scores| < 100, d <= 128).

Gradients. The kernels round P (u), dS (u), o (u, through D = dout . o) and the result (u), and
the sums behind a result add these errors: |dv| error <= u sum |P dout| + u |dv|, |dk| error <=
scale (u sum |dS q| + ...): see grad_bounds, which evaluates these sums in 64 bits.
"""
import math

import numpy as np
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
