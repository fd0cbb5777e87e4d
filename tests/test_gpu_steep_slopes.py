"""Distance slopes of every size and sign: a key beside the query gets its logit
to fp32's precision, however steeply the far keys of its tile fall off."""
import math

import pytest
import torch

import _mod_ref as R
import _rows
from attention_forward_online_gb300 import osattn

pytestmark = pytest.mark.gpu
DEV, F64 = "cuda", torch.float64
BF, FP = torch.bfloat16, torch.float16

SLOPES = [-3.0, -0.25, 0.0, 0.7, 1.0, 8.0, 32.0, 1400.0]
# Slopes of at most 1 may enter through the tensor core: score and slope / scale
# times a place below 128 are added in fp32, off by at most 2^-23 of 128 slopes
# an addition, of which there are two (and the constant that is taken off again).
LINEAR = 3 * 2.0 ** -23 * 128


def bias_and_error(gap):
    s = torch.tensor(SLOPES, dtype=F64, device=DEV)[:, None, None]
    return -s * gap.abs(), torch.where(s.abs() <= 1, LINEAR * s.abs(), torch.zeros_like(s))


@pytest.mark.parametrize("dtype,d", [(BF, 64), (BF, 128), (FP, 64), (FP, 128)],
                         ids=["bf16-64", "bf16-128", "fp16-64", "fp16-128"])
@pytest.mark.parametrize("scale", [None, 2.0, -0.01])
@pytest.mark.parametrize("causal", [True, False])
def test_dense(causal, scale, dtype, d):
    B, H, N = 1, len(SLOPES), 333
    g = torch.Generator(device=DEV).manual_seed(d)
    q, k, v, do = (torch.randn(B, H, N, d, generator=g, device=DEV).to(dtype) for _ in range(4))
    slopes = torch.tensor(SLOPES, device=DEV)
    plan = osattn.mask_plan(B, N, N, causal=causal, device=DEV)
    o, lse = osattn.fwd_mod(q, k, v, scale, plan=plan, slopes=slopes)
    grads = osattn.bwd_mod(q, k, v, o, lse, do, scale, plan=plan, slopes=slopes)
    assert osattn.get_device_status() == osattn.OK
    sc = 1 / math.sqrt(d) if scale is None else scale
    gap = R.distance(N, N, device=DEV)
    see = (gap <= 0) if causal else torch.ones_like(gap, dtype=torch.bool)
    bias, linear = bias_and_error(gap)
    qq, kk, vv = (x.to(F64) for x in (q, k, v))
    y = sc * (qq @ kk.transpose(-1, -2))
    err = _rows.score_error(qq, kk, sc, y, bias) + linear
    _rows.check({"o": o, "lse": lse}, _rows.rows(y + bias, see, err, vv, dtype))
    want = R.reference(q, k, v, see[None], sc, do, 0.0, slopes)
    for name, got in zip(("dq", "dk", "dv"), grads):
        # (the bounds of R.reference are for slopes that are not negative; for
        # the two others the error's norm: four roundings of half a step)
        R.check(got[:, 2:], want[name][0][:, 2:], want[name][1][:, 2:], name)
        val = want[name][0][:, :2]
        assert float((got[:, :2].to(F64) - val).norm() / val.norm()) < 4 * R.U[dtype]


@pytest.mark.parametrize("dtype,d", [(BF, 128), (FP, 64)], ids=["bf16-128", "fp16-64"])
@pytest.mark.parametrize("T", [1, 5])
def test_over_a_cache(T, dtype, d):
    B, H, page, ctx = 1, len(SLOPES), 16, 300
    g = torch.Generator(device=DEV).manual_seed(d + T)
    per = -(-(ctx + T) // page)
    q = torch.randn(B, H, T, d, generator=g, device=DEV).to(dtype)
    for Hkv in (H, 2):
        kp, vp = (torch.randn(per, Hkv, page, d, generator=g, device=DEV).to(dtype) for _ in range(2))
        table = torch.arange(per, dtype=torch.int32, device=DEV).reshape(1, per)
        o, lse = osattn.tree_attn(q, kp, vp, table, torch.full((1,), ctx, dtype=torch.int32, device=DEV),
                                  slopes=torch.tensor(SLOPES, device=DEV))
        n = ctx + T
        kk, vv = (x.transpose(0, 1).reshape(1, Hkv, per * page, d)[:, :, :n].to(F64).repeat_interleave(H // Hkv, 1)
                  for x in (kp, vp))
        gap = torch.arange(n, device=DEV)[None] - ctx - torch.arange(T, device=DEV)[:, None]
        bias, linear = bias_and_error(gap)
        sc, qq = 1 / math.sqrt(d), q.to(F64)
        y = sc * (qq @ kk.transpose(-1, -2))
        err = _rows.score_error(qq, kk, sc, y, bias) + linear
        _rows.check({"o": o, "lse": lse}, _rows.rows(y + bias, gap <= 0, err, vv, dtype))
