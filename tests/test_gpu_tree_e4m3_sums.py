"""Tree attention over e4m3 pages: sums of weights over V scales at the ends of their
range, in shares of many keys.  Sequences share their pages, so that every CTA has a
unit as long as the longest context; both forms (3 drafts of 4 heads: few rows, 9: many).

All keys of the context have one logit, the drafts a lower one, which is that of
the first keys that a share takes.  The kernels add up a row's sum of n equal terms a thread, at most 2^-24 of the
sum an addition, 16 additions a tile: |d sum| <= 16 tiles 2^-24 of it; a weight is off by 2^-22
and rounded to fp16's 2^-11 for the product with V, and the logit by 8 steps of 2^-24 of
the largest of its numbers."""
import math

import pytest
import torch

import _cache_ref as R
from attention_forward_online_gb300 import osattn

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF, FP, E4 = torch.bfloat16, torch.float16, torch.float8_e4m3fn
FEW, MANY = 3, 9
D, PAGE, H = 64, 128, 4


def shared(B, ctx, T, high, low, v_scale, dtype, zero=True):
    """B sequences of the same ctx keys of logit `high` and T drafts of logit `low` (e4m3 values)."""
    n = -(-(ctx + T) // PAGE)
    g = torch.Generator(device=DEV).manual_seed(ctx)
    k = torch.zeros(n, 1, PAGE, D, device=DEV)
    k[..., 0] = high
    k.view(-1, D)[ctx:, 0] = low
    v = torch.randn(n, 1, PAGE, D, generator=g, device=DEV) * (0 if zero else 64)
    q = torch.zeros(B, H, T, D, dtype=dtype, device=DEV)
    q[..., 0] = 1.0
    return dict(q=q, k=k.to(E4), v=(v + (0 if zero else 100)).clamp(-448, 448).to(E4), ks=torch.ones(n, 1, 1, device=DEV),
                vs=torch.full((n, 1, 1), v_scale, device=DEV),
                table=torch.arange(n, dtype=torch.int32, device=DEV)[None].expand(B, n).contiguous(),
                ctx=torch.full((B,), ctx, dtype=torch.int32, device=DEV))


def call(s):
    o, lse = osattn.tree_attn(s["q"], s["k"], s["v"], s["table"], s["ctx"], scale=1.0, k_scale=s["ks"], v_scale=s["vs"])
    assert osattn.get_device_status() == osattn.OK
    return o, lse


def check(s, ctx, T, high, low):
    o, lse = call(s)
    tiles = -(-(ctx + T) // 128)
    # draft t sees the context and drafts 0 .. t
    weights = torch.full((T, ctx + T), 0.0, dtype=torch.float64)
    weights[:, :ctx] = math.exp(high - low)
    weights[:, ctx:] = torch.tril(torch.ones(T, T))
    total = weights.sum(1)
    want = (low + total.log()).to(DEV)
    sums = 16 * tiles * 2.0 ** -24 + 2.0 ** -21
    assert torch.isfinite(lse).all()
    off = (lse.double() - want).abs()
    assert (off <= sums + 8 * 2.0 ** -24 * (abs(high) + want.abs())).all(), float(off.max())
    v = R.dequantised(s["v"], s["vs"])[:, 0].reshape(-1, D)[:ctx + T]
    p = (weights / total[:, None]).to(DEV)
    mean, size = p @ v, p @ v.abs()
    lim = (2.0 ** -11 + 2 * sums + 16 * 2.0 ** -24 * abs(high)) * size + R.U[o.dtype] * mean.abs() + R.TINY[o.dtype]
    off = (o.double() - mean).abs()
    assert (off <= lim).all(), float((off / lim.clamp(min=1e-300)).max())


@pytest.mark.parametrize("T", [FEW, MANY])
@pytest.mark.parametrize("B", [152, 100], ids=["whole", "cut"])
def test_values_of_zero_behind_a_lower_first_tile(B, T):
    # e^3.9375 = 2^5.68: m stays at the drafts' level, weights over s_v are 2^(15.68 + 100)
    check(shared(B, 32768, T, 4.0, 0.0625, 2.0 ** -100, BF), 32768, T, 4.0, 0.0625)


@pytest.mark.parametrize("T", [FEW, MANY])
def test_values_of_zero_and_equal_scores_of_a_long_context(T):
    check(shared(152, 400000, T, 0.0, 0.0, 0.0, FP), 400000, T, 0.0, 0.0)


@pytest.mark.parametrize("T", [FEW, MANY])
@pytest.mark.parametrize("exponent", [-100, -40, 0, 60, 104, 112, 119])
def test_values_of_any_scale(exponent, T):
    check(shared(100, 32768, T, 4.0, 0.0625, 2.0 ** exponent, BF, zero=False), 32768, T, 4.0, 0.0625)
