"""Norms of rows whose squares leave FP32: infinitely long, they become zeros, whatever the weight, and so
do their gradients; the rows beside them keep theirs. Bounds of the others as in _cache8.py."""
import pytest
import torch

import _cache8 as c8
import tiled_attention_06_gb300 as fa

pytestmark = pytest.mark.gpu
BF, HF, FP = torch.bfloat16, torch.float16, torch.float32
SIZES = (1e20, 3e38, -3e38)


def rows(T, H, d, dtype, seed):
    """Token 1's rows are of the largest finite sizes, each element of a token's head the same."""
    x = torch.randn(T, H, d, generator=torch.Generator().manual_seed(seed))
    for h in range(H):
        x[1, h] = SIZES[h % len(SIZES)]
    x[2, 0, 3] = 3e38  # one such element is enough
    return x.to(dtype)


@pytest.mark.parametrize("dtype,wdt", [(BF, BF), (BF, FP), (FP, FP)], ids=str)
@pytest.mark.parametrize("d,half", [(64, True), (128, False), (6, True)])
def test_infinitely_long_rows_become_zeros(dtype, wdt, d, half):
    T, H = 5, 3
    x = rows(T, H, d, dtype, 1)
    w = (2 + torch.rand(d, generator=torch.Generator().manual_seed(2))).to(wdt)  # w x alone leaves FP32
    dy = torch.randn(T, H, d, generator=torch.Generator().manual_seed(3)).to(dtype)
    pos, freqs = torch.arange(T, dtype=torch.int32), fa.fa_rope_freqs(d)[0]
    args = (pos[None], torch.zeros(d // 2), freqs, d, half)
    y, dx = (torch.full((T, H, d), 7.0, dtype=dtype, device="cuda") for _ in range(2))
    dw = torch.empty(d, device="cuda")
    ws = torch.empty(fa.fa_norm_rope_bwd_workspace_size(H, 0, d), dtype=torch.uint8, device="cuda")
    kw = dict(q_weight=w.cuda(), norm=fa.FA_NORM_RMS, style=fa.FA_ROPE_HALF if half else fa.FA_ROPE_PAIRS)
    fa.fa_norm_rope(x.cuda(), None, y, None, pos.cuda(), freqs.cuda(), **kw)
    fa.fa_norm_rope_bwd(x.cuda(), None, dy.cuda(), None, dx, None, pos.cuda(), freqs.cuda(), dq_weight=dw,
                        workspace=ws, **kw)
    torch.cuda.synchronize()
    assert fa.fa_get_device_status() == fa.FA_OK
    gone = torch.zeros(T, H, dtype=torch.bool)
    gone[1], gone[2, 0] = True, True
    for got in (y.cpu(), dx.cpu()):
        assert (got[gone] == 0).all()
    # the others, as if those were not there: a row of zeros has neither output nor part in the sum
    x, dy = (torch.where(gone[..., None], torch.zeros((), dtype=dtype), t) for t in (x, dy))
    want, bound = c8.norm_rope(x, w, 1e-6, *args)
    c8.check(y, want, bound, dtype, "y")
    (gx, bx), (gw, bw) = c8.norm_rope_grad(x, w, 1e-6, dy, *args)
    c8.check(dx, gx, bx, dtype, "dx")
    c8.check(dw, gw, bw, FP, "dw")


@pytest.mark.parametrize("bits", [8, 16])
def test_infinitely_long_keys_in_the_cache(bits):
    T, d, page = 4, 64, 16
    x = rows(T, 2, d, BF, 4)
    w = torch.full((d,), 2.5, dtype=BF)
    i32 = dict(dtype=torch.int32, device="cuda")
    shape = (1, 1, page, d)
    pools = [torch.full(shape, 9, dtype=torch.uint8, device="cuda") if bits == 8 else
             torch.full(shape, 7.0, dtype=BF, device="cuda") for _ in range(2)]
    kw = {n: torch.full(shape[:3], 9, dtype=torch.uint8, device="cuda")
          for n in ("k_scales", "v_scales")} if bits == 8 else {}
    q_out = torch.empty(T, 1, d, dtype=BF, device="cuda")
    dev = x.cuda()
    v = torch.ones(T, 1, d, dtype=BF, device="cuda")
    fa.fa_norm_rope_append(dev[:, :1], dev[:, 1:], v, q_out, *pools, torch.zeros(1, 1, **i32),
                           torch.zeros(1, **i32), torch.tensor([0, T], **i32), fa.fa_rope_freqs(d)[0].cuda(),
                           q_weight=w.cuda(), k_weight=w.cuda(), norm=fa.FA_NORM_RMS, **kw)
    torch.cuda.synchronize()
    assert fa.fa_get_device_status() == fa.FA_OK
    assert (q_out[1:3] == 0).all() and torch.isfinite(q_out.float()).all()
    k = pools[0][0, 0, :T].cpu()
    if bits == 8:
        e = kw["k_scales"][0, 0, :T].cpu()
        assert e[1] == 0 and (e != 255).all()
        k = c8.values(k, e)
    assert (k[1] == 0).all() and torch.isfinite(k.float()).all() and (k[0] != 0).any()
