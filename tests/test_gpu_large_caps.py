"""Capped scores far below their cap are good to fp32's relative precision in
every path, whatever the cap's size: an absolute error that grows with the cap
would be 2e-3 in a logit at a cap of 10^4."""
import math

import pytest
import torch

import _rows
from attention_forward_online_gb300 import osattn

pytestmark = pytest.mark.gpu
DEV, F64 = "cuda", torch.float64
BF, FP = torch.bfloat16, torch.float16
TYPES = pytest.mark.parametrize("dtype,d", [(BF, 128), (FP, 64)], ids=["bf16-128", "fp16-64"])


def slopes_of(H):
    return torch.exp2(-8.0 * torch.arange(1, H + 1, device=DEV, dtype=torch.float32) / H)


@pytest.mark.parametrize("cap", [1e3, 1e4])
@pytest.mark.parametrize("sloped", [False, True])
@pytest.mark.parametrize("shape", [(1, 2, 1, 3, 5), (2, 4, 2, 150, 150), (1, 2, 2, 40, 300)],
                         ids=lambda s: "x".join(map(str, s)))
@TYPES
def test_dense(shape, sloped, cap, dtype, d):
    B, H, Hkv, Nq, Nkv = shape
    g = torch.Generator(device=DEV).manual_seed(Nkv + d)
    q = (torch.randn(B, H, Nq, d, generator=g, device=DEV) * 2).to(dtype)
    k, v = (torch.randn(B, Hkv, Nkv, d, generator=g, device=DEV).to(dtype) for _ in range(2))
    slopes = slopes_of(H) if sloped else None
    off = Nkv - Nq
    for masks in ({}, dict(causal=True), dict(causal=True, window=9)):
        plan = osattn.mask_plan(B, Nq, Nkv, q_offset=off, device=DEV, **masks)
        o, lse = osattn.fwd_mod(q, k, v, plan=plan, softcap=cap, slopes=slopes)
        assert osattn.get_device_status() == osattn.OK
        qq, kk, vv = (x.to(F64) for x in (q, k.repeat_interleave(H // Hkv, 1), v.repeat_interleave(H // Hkv, 1)))
        gap = (torch.arange(Nkv, device=DEV)[None] - torch.arange(Nq, device=DEV)[:, None] - off)
        see = torch.ones(Nq, Nkv, dtype=torch.bool, device=DEV)
        if masks:
            see &= gap <= 0
        if "window" in masks:
            see &= gap.abs() < masks["window"]
        bias = torch.zeros(H, 1, 1, dtype=F64, device=DEV) if slopes is None else -slopes.to(F64)[:, None, None] * gap.abs()
        scale = 1 / math.sqrt(d)
        y = _rows.capped(scale * (qq @ kk.transpose(-1, -2)), cap)
        assert float(y.abs().max()) < 0.2 * cap
        err = _rows.score_error(qq, kk, scale, y, bias)
        _rows.check({"o": o, "lse": lse}, _rows.rows(y + bias, see, err, vv, dtype))


@pytest.mark.parametrize("cap", [1e3, 1e4])
@pytest.mark.parametrize("sloped", [False, True])
@pytest.mark.parametrize("T,ctx,window", [(1, 4, 0), (1, 300, 0), (6, 130, 0), (9, 500, 40)])
@TYPES
def test_over_a_cache(T, ctx, window, sloped, cap, dtype, d):
    B, H, Hkv, page = 2, 4, 2, 16
    g = torch.Generator(device=DEV).manual_seed(ctx + T)
    per = -(-(ctx + T) // page)
    q = (torch.randn(B, H, T, d, generator=g, device=DEV) * 2).to(dtype)
    kp, vp = (torch.randn(B * per, Hkv, page, d, generator=g, device=DEV).to(dtype) for _ in range(2))
    table = torch.arange(B * per, dtype=torch.int32, device=DEV).flip(0).reshape(B, per)
    slopes = slopes_of(H) if sloped else None
    o, lse = osattn.tree_attn(q, kp, vp, table, torch.full((B,), ctx, dtype=torch.int32, device=DEV),
                              softcap=cap, slopes=slopes, window=window)
    assert osattn.get_device_status() == osattn.OK
    n = ctx + T
    kk, vv = (x[table.long()].transpose(1, 2).reshape(B, Hkv, per * page, d)[:, :, :n].to(F64)
              .repeat_interleave(H // Hkv, 1) for x in (kp, vp))
    gap = torch.arange(n, device=DEV)[None] - ctx - torch.arange(T, device=DEV)[:, None]
    see = gap <= 0
    if window:
        see &= gap > -window
    bias = torch.zeros(H, 1, 1, dtype=F64, device=DEV) if slopes is None else -slopes.to(F64)[:, None, None] * gap.abs()
    scale, qq = 1 / math.sqrt(d), q.to(F64)
    y = _rows.capped(scale * (qq @ kk.transpose(-1, -2)), cap)
    assert float(y.abs().max()) < 0.2 * cap
    err = _rows.score_error(qq, kk, scale, y, bias)
    _rows.check({"o": o, "lse": lse}, _rows.rows(y + bias, see, err, vv, dtype))


@pytest.mark.parametrize("dtype,d", [(BF, 64), (BF, 128), (FP, 64), (FP, 128)],
                         ids=["bf16-64", "bf16-128", "fp16-64", "fp16-128"])
def test_scores_on_both_sides_of_the_border(dtype, d):
    # rows whose scores stay far below the cap beside rows that saturate it:
    # the form changes from block to block, and masked places decide nothing
    B, H, N, cap = 1, 4, 400, 3.0
    g = torch.Generator(device=DEV).manual_seed(5)
    q = (torch.randn(B, H, N, d, generator=g, device=DEV) * 0.2).to(dtype)
    q[:, :, 150:190] *= 40
    k, v = (torch.randn(B, H, N, d, generator=g, device=DEV).to(dtype) for _ in range(2))
    slopes = slopes_of(H)
    plan = osattn.mask_plan(B, N, N, causal=True, window=170, device=DEV)
    o, lse = osattn.fwd_mod(q, k, v, plan=plan, softcap=cap, slopes=slopes)
    k2 = k.clone()
    gap = torch.arange(N, device=DEV)[None] - torch.arange(N, device=DEV)[:, None]
    see = (gap <= 0) & (gap > -170)
    scale = 1 / math.sqrt(d)
    qq, kk, vv = (x.to(F64) for x in (q, k, v))
    y = _rows.capped(scale * (qq @ kk.transpose(-1, -2)), cap)
    bias = -slopes.to(F64)[:, None, None] * gap.abs()
    # where the cap bends scores: within 2^-20 of the cap, see osattn.h
    err = _rows.score_error(qq, kk, scale, y, bias) + 2.0 ** -20 * cap
    _rows.check({"o": o, "lse": lse}, _rows.rows(y + bias, see, err, vv, dtype))
    # keys that a query does not see may hold anything
    k2[:, :, 390:] = math.inf
    plan = osattn.mask_plan(B, N, N, causal=True, key_len=torch.full((1,), 390, dtype=torch.int32, device=DEV))
    one = osattn.fwd_mod(q, k, v, plan=plan, softcap=cap, slopes=slopes)
    two = osattn.fwd_mod(q, k2, v, plan=plan, softcap=cap, slopes=slopes)
    assert torch.equal(one[0], two[0]) and torch.equal(one[1], two[1])
