"""How near rotations and attention over e4m3 pages are to 64 bits, by what the kernels'
arithmetic can lose: tighter than _cache_ref.py's bounds, which hold for any inputs.

Sines and cosines: the polynomials in fp32, over all phases, are within 5.8e-8 of the sine and
7.6e-8 of the cosine of an angle of at most an eighth of a turn (1.44e-8 and 1.91e-8 rms, by
evaluating them on a CPU with exact sums rounded once); the angle is cut to 2^-32 turns,
1.5e-9 radians.

A rotation multiplies each by the amplitude, and rounds a product and a sum:
  |dy| <= m (|a| + |b|) (7.6e-8 + 1.5e-9 + 2 2^-24 + p f 2^-51) + 2^-24 |y|, and the type's rounding.

Attention: the elements of a query are in two or three 8-bit terms to 2^-21 of their row's greatest,
the tensor cores add products to 2^-21 of the sum of their magnitudes (the second and third
terms add a sixteenth), a logit takes 8 steps of 2^-24 more, and weights are rounded to
fp16.  So LSE is as near as its logits,
  |dLSE| <= scale 2^-21 (max |q| sum |k| + 17/16 ||q|| ||k||) + 8 2^-24 max |y| + 2^-19 (sums) + 2^-22 |LSE|
and of the output's size O is off by its own rounding and the weights', as independent errors: values
of any size within their binade are rounded off by 0.425 of half a step, rms."""
import math

import pytest
import torch

import _cache_ref as R
from attention_forward_online_gb300 import osattn
from test_gpu_tree_e4m3 import BF, DEV, FP, run, setup, slopes_of

pytestmark = pytest.mark.gpu
F32 = torch.float32


def test_sines_and_cosines():
    N, half = 1 << 16, 64
    q = torch.zeros(1, 1, N, 2 * half, device=DEV)
    q[..., :half] = 1.0  # pairs (1, 0) become (cos, sin)
    f = osattn.rotary_freqs(2 * half, base=3.7e4).to(DEV) + 0.013
    at = torch.randint(0, 1 << 20, (N,), generator=torch.Generator().manual_seed(1)).int().to(DEV)
    got = osattn.rotary(q, freqs=f, positions=at)[0, 0].double()
    t = at.double()[:, None] * f
    want = torch.cat([torch.cos(t), torch.sin(t)], 1)
    off = (got - want).abs()
    slack = 1.5e-9 + float(t.max()) * 2.0 ** -51
    near = want.abs() < math.sqrt(0.5)  # a sine of the distance from a quarter turn
    assert float(off[near].max()) <= 5.8e-8 + slack and float(off[~near].max()) <= 7.6e-8 + slack
    assert float((off[near] ** 2).mean().sqrt()) <= 1.2 * 1.44e-8
    assert float((off[~near] ** 2).mean().sqrt()) <= 1.2 * 1.91e-8


@pytest.mark.parametrize("inverse", [False, True])
@pytest.mark.parametrize("interleaved", [False, True], ids=["halves", "pairs"])
@pytest.mark.parametrize("dtype", [BF, FP, F32], ids=["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("d,rot", [(128, 128), (80, 20), (64, 48)])
def test_rotations(d, rot, dtype, interleaved, inverse):
    g = torch.Generator(device=DEV).manual_seed(rot)
    q = torch.randn(2, 3, 500, d, generator=g, device=DEV).to(dtype)
    at = torch.randint(0, 1 << 20, (500,), generator=g, device=DEV).int()
    f = osattn.rotary_freqs(rot).to(DEV)
    m = 1.3
    got = osattn.rotary(q, freqs=f, positions=at, interleaved=interleaved, amplitude=m, inverse=inverse)
    want, _ = R.rotate(q, at, f, interleaved, m, inverse)
    x = q.double()
    i = torch.arange(rot // 2, device=DEV)
    first, second = (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)
    off = torch.zeros_like(want)
    t = at.double()[:, None] * f
    off[..., first] = off[..., second] = m * (x[..., first].abs() + x[..., second].abs()) * (
        7.6e-8 + 1.5e-9 + 2.0 ** -23 + t * 2.0 ** -51)
    off[..., :rot] += 2.0 ** -24 * want[..., :rot].abs()
    if dtype is not F32:
        off = R.stored(want, off, dtype)
    err = (got.double() - want).abs()
    assert (err <= off).all(), float((err / off.clamp(min=1e-300)).max())


@pytest.mark.parametrize("kind", ["plain", "cap", "slopes"])
@pytest.mark.parametrize("T", [1, 4, 9, 32])
@pytest.mark.parametrize("dtype,d", [(BF, 128), (FP, 64), (BF, 64), (FP, 128)],
                         ids=["bf16-128", "fp16-64", "bf16-64", "fp16-128"])
def test_attention(dtype, d, T, kind):
    kw = {"plain": {}, "cap": dict(cap=20.0), "slopes": dict(slopes=slopes_of(8))}[kind]
    ctx = [3000, 777]
    s = setup(2, 8, 2, T, d, 64, 64, ctx, dtype, seed=T + d)
    scale = 1 / math.sqrt(d)
    got = run(s, softcap=kw.get("cap", 0.0), slopes=kw.get("slopes"), scale=scale)
    ref = R.tree8_reference(s["q"], s["k"], s["v"], s["ks"], s["vs"], s["table"], ctx, s["masks"], scale,
                            kw.get("cap", 0.0), kw.get("slopes"), 0)
    want = ref["o"][0]
    size = want.norm()
    own = float((want.to(dtype).double() - want).norm() / size)
    off = float((got["o"].double() - want).norm() / size)
    assert off <= 1.15 * math.hypot(own, 0.425 * 2.0 ** -11), (off, own)
    k = R.dequantised(s["k"], s["ks"])
    lse = ref["lse"][0]
    for b in range(2):
        keys = torch.arange(ctx[b] + T, device=DEV)
        kk = k[s["table"][b].long()[keys // 64], :, keys % 64]  # [n, Hkv, d]
        q = s["q"][b].double()
        most = kk.norm(dim=-1).amax(0).repeat_interleave(4)[:, None]
        sums = kk.abs().sum(-1).amax(0).repeat_interleave(4)[:, None]
        y = scale * q.norm(dim=-1) * most + (ctx[b] * slopes_of(8)[:, None] if kind == "slopes" else 0.0)
        lim = scale * 2.0 ** -21 * (q.abs().amax(-1) * sums + 17 / 16 * q.norm(dim=-1) * most)
        lim = lim + 2.0 ** -21 * y + 2.0 ** -19 + 2.0 ** -22 * lse[b].abs()
        if kind == "cap":
            lim = lim + 2.0 ** -20 * 20.0  # the cap itself
        err = (got["lse"][b].double() - lse[b]).abs()
        assert (err <= lim).all(), float((err / lim).max())
