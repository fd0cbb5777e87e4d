"""Tree attention over e4m3 pages: many keys far below a row's greatest, which weigh something
together.  Every CTA has such a key in its even and in its odd tiles, and its values
are zeros, so that the result is the others'.

A weight x is an fp16 value, the greatest 2^10 of its row: off by 2^-11 of itself or 2^-25.
It is three e5m2 terms, whose least step is 2^-16.  With few rows the second counts 2^-3 and the
last 2^-7: what is left of x behind the second is at most 2^-20 where that is a subnormal, the last
term's steps are 2^-23 there, so 1.5 2^-24 is lost, 1.5 2^-34 of the greatest:
  |dO| <= sum (2^-11 P + 1.5 2^-34) |V|
With many rows the terms are one sum, and a weight is off by 2^-17, half the least step (half of it once
more where the second term rounds a remainder of 2^-17 up):
  |dO| <= sum (2^-11 P + 2^-26) |V|
with P relative to the greatest; besides, the logits' and sums' errors (see test_gpu_tree_e4m3_sums)."""
import math

import pytest
import torch

import _cache_ref as R
from attention_forward_online_gb300 import osattn

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF, FP, E4 = torch.bfloat16, torch.float16, torch.float8_e4m3fn
FEW, MANY = 3, 9
D, PAGE, H, B, CTX = 64, 128, 4, 152, 102400


@pytest.mark.parametrize("T", [FEW, MANY])
@pytest.mark.parametrize("dtype", [BF, FP], ids=["bf16", "fp16"])
@pytest.mark.parametrize("bits", [20, 25.5, 26.5, 28, 31, 33])
def test_many_keys_far_below_the_greatest(bits, dtype, T):
    n = CTX // PAGE + 1
    k = torch.zeros(n * PAGE, D, device=DEV)
    k[CTX - 1:, 0] = 448.0  # a key of the context's last tile, and the drafts
    v = torch.zeros(n * PAGE, D, device=DEV)
    g = torch.Generator(device=DEV).manual_seed(1)
    v[:CTX - 1] = (100 + 20 * torch.randn(CTX - 1, D, generator=g, device=DEV)).clamp(1, 448)
    k, v = (x.to(E4).reshape(n, 1, PAGE, D) for x in (k, v))
    scales = torch.ones(n, 1, 1, device=DEV)
    q = torch.zeros(B, H, T, D, dtype=dtype, device=DEV)
    q[..., 0] = 1.0
    scale = bits * math.log(2) / 448
    o, lse = osattn.tree_attn(q, k, v, torch.arange(n, dtype=torch.int32, device=DEV)[None].expand(B, n),
                              torch.full((B,), CTX, dtype=torch.int32, device=DEV), scale=scale, k_scale=scales,
                              v_scale=scales)
    assert osattn.get_device_status() == osattn.OK
    above = (torch.arange(T, dtype=torch.float64) + 2).to(DEV)  # keys at the top: the last cached one and drafts 0 .. t
    total = above + (CTX - 1) * 2.0 ** -bits
    mean = v.double().reshape(-1, D)[:CTX - 1].mean(0) * (CTX - 1) * 2.0 ** -bits / total[:, None]
    sums = 16 * n * 2.0 ** -24 + 2.0 ** -21 + 16 * 2.0 ** -24 * bits
    off = (lse.double() - (bits * math.log(2) + total.log())).abs()
    assert (off <= sums + 16 * 2.0 ** -24 * bits).all(), float(off.max())
    size = v.double().reshape(-1, D)[:CTX - 1].sum(0) / total[:, None]
    small = 2.0 ** -11 * mean + (1.5 * 2.0 ** -34 if T == FEW else 2.0 ** -26) * size
    lim = small + 2 * sums * mean + R.U[dtype] * mean + R.TINY[dtype]
    off = (o.double() - mean).abs()
    assert (off <= lim).all(), (float((off / lim).max()), float(o.double().mean() / mean.mean()))
