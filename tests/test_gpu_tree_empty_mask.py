"""A draft whose mask is empty stands one place before the context's end (bits of
its mask - 1) for the drafts that see it, as every draft stands by its own mask."""
import math

import pytest
import torch

import _rows
from attention_forward_online_gb300 import osattn

pytestmark = pytest.mark.gpu
DEV, F64 = "cuda", torch.float64


@pytest.mark.parametrize("dtype,d", [(torch.bfloat16, 128), (torch.float16, 64)], ids=["bf16-128", "fp16-64"])
@pytest.mark.parametrize("window", [0, 1, 2, 3, 4])
@pytest.mark.parametrize("sloped", [False, True])
def test_drafts_that_see_an_empty_one(sloped, window, dtype, d):
    B, H, page, T = 2, 4, 16, 3
    ctxs, masks = [40, 3], [[1, 0, 7], [0, 3, 1]]
    g = torch.Generator(device=DEV).manual_seed(d)
    per = 3
    kp, vp = (torch.randn(B * per, H, page, d, generator=g, device=DEV).to(dtype) for _ in range(2))
    table = torch.arange(B * per, dtype=torch.int32, device=DEV).reshape(B, per)
    q = torch.randn(B, H, T, d, generator=g, device=DEV).to(dtype)
    slopes = torch.tensor([0.9, 0.5, 0.3, 0.1], device=DEV) if sloped else None
    o, lse = osattn.tree_attn(q, kp, vp, table, torch.tensor(ctxs, dtype=torch.int32, device=DEV),
                              torch.tensor(masks, device=DEV), slopes=slopes, window=window)
    assert osattn.get_device_status() == osattn.OK
    for b, ctx in enumerate(ctxs):
        n = ctx + T
        pos = torch.tensor([ctx + bin(m).count("1") - 1 for m in masks[b]], device=DEV)
        at = torch.cat([torch.arange(ctx, device=DEV), pos])
        gap = (pos[:, None] - at[None]).abs()
        see = torch.zeros(T, n, dtype=torch.bool, device=DEV)
        for t, m in enumerate(masks[b]):
            see[t, :ctx] = m != 0
            for x in range(T):
                see[t, ctx + x] = bool((m >> x) & 1)
        if window:
            see &= gap < window
        kk, vv = (x[table[b].long()].transpose(0, 1).reshape(H, per * page, d)[:, :n].to(F64) for x in (kp, vp))
        bias = torch.zeros(H, 1, 1, dtype=F64, device=DEV)
        if sloped:
            bias = -slopes.to(F64)[:, None, None] * gap
        scale, qq = 1 / math.sqrt(d), q[b].to(F64)
        y = scale * (qq @ kk.transpose(-1, -2))
        err = _rows.score_error(qq, kk, scale, y, bias)
        _rows.check({"o": o[b], "lse": lse[b]}, _rows.rows(y + bias, see, err, vv, dtype))
