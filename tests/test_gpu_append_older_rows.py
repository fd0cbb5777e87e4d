"""The older rows of a block that an append adds to (osattn_cache_append, e4m3 pages): as
they were where the block keeps its scale, rounded once to a greater one, whether a warp
(16 new tokens or fewer) or a thread block takes the unit, and for scales that
say nothing."""
import math

import pytest
import torch

import _cache_ref as R
from attention_forward_online_gb300 import osattn
from test_gpu_append import BF, DEV, E4, FP, Cache, untouched

pytestmark = pytest.mark.gpu


def codes(c, x, b, lo, hi):
    """Rows lo .. hi of sequence b, [Hkv, n, d] bytes."""
    at = torch.arange(lo, hi, device=DEV)
    return x.view(torch.uint8)[c.table[b].long()[at // c.page], :, at % c.page].transpose(0, 1).contiguous()


def check_older(c, before, b, ctx, count, block, new):
    """The older rows of the block that ctx falls into, and the block's scale; `new` [K and V rows of it, or None]."""
    lo = ctx // block * block
    kept = grown = 0
    for x, s, was, f, rows in ((c.k, c.ks, before[0], before[2], new[0]), (c.v, c.vs, before[1], before[3], new[1])):
        had, has = (c.factors(y, b, lo, lo + 1)[:, 0] for y in (f, s))
        if rows is not None:
            assert torch.equal(has, torch.maximum(had, R.power(R.scale_exponent(rows.double().abs().amax((1, 2))))))
        old, now = codes(c, was, b, lo, ctx), codes(c, x, b, lo, ctx)
        for h in range(len(had)):
            if has[h] == had[h]:
                kept += 1
                assert torch.equal(old[h], now[h])
            else:
                grown += 1
                assert has[h] > had[h]
                want = (old[h].view(E4).double() * (had[h] / has[h])).float().to(E4).double()
                got = now[h].view(E4).double()
                assert ((got == want) | (got.isnan() & want.isnan())).all()
    return kept, grown


# d, page, block, ctx: blocks longer and shorter than the rows that a unit's registers hold
BLOCKS = [(64, 32, 8, [3, 39, 700]), (128, 64, 64, [1, 100, 63]), (128, 256, 128, [100, 383, 129]),
          (64, 512, 256, [255, 300, 1]), (128, 384, 384, [200, 385, 300])]


@pytest.mark.parametrize("turned", [False, True], ids=["as-they-are", "turned"])
@pytest.mark.parametrize("T", [1, 16, 17, 64, 300])
@pytest.mark.parametrize("d,page,block,ctx", BLOCKS)
def test_older_rows_stay_or_are_rounded_once(d, page, block, ctx, T, turned):
    B, Hkv = 3, 4
    dtype = BF if T % 2 else FP
    c = Cache(B, Hkv, d, page, max(ctx) + T, dtype, block, seed=T, layout="pshd" if T % 3 == 0 else "phsd")
    g = torch.Generator(device=DEV).manual_seed(T + d)
    for s in (c.ks, c.vs):  # the new rows need 2^-8 or so: some blocks grow and some do not
        s.copy_(torch.exp2(torch.randint(-13, -2, s.shape, generator=g, device=DEV).float()))
    k, v = (torch.randn(B, Hkv, T, d, generator=g, device=DEV).to(dtype) for _ in range(2))
    raw = c.copies()
    before = [x.view(E4) if x.dtype == torch.uint8 else x for x in raw]
    c.append(k, v, ctx, **(dict(freqs=osattn.rotary_freqs(d // 2).to(DEV)) if turned else {}))
    kept = grown = 0
    for b in range(B):
        n = min(T, (ctx[b] // block + 1) * block - ctx[b])
        if ctx[b] % block:
            x = check_older(c, before, b, ctx[b], T, block, (None if turned else k[b, :, :n], v[b, :, :n]))
            kept, grown = kept + x[0], grown + x[1]
    assert kept and grown  # both happened
    untouched(c, raw, B, ctx, [T] * B)


@pytest.mark.parametrize("T", [1, 17])
def test_older_rows_of_a_scale_of_zero_are_zeros(T):
    # as the attention call reads them, before and after
    c = Cache(1, 2, 64, 64, 128, BF, 64)
    k, v = (torch.ones(1, 2, T, 64, dtype=BF, device=DEV) for _ in range(2))
    for x in (c.k, c.v):
        raw = x.view(torch.uint8)
        raw[(raw & 0x7f) == 0x7f] = 0x30
    for s in (c.ks, c.vs):
        s.zero_()
    c.append(k, v, [40])
    for x, s in ((c.k, c.ks), (c.v, c.vs)):
        assert (c.factors(s, 0, 0, 1) == 2.0 ** -8).all()
        assert not c.rows(x, 0, 0, 40).any()
        assert (c.rows(x, 0, 40, 40 + T) == 256.0).all()


@pytest.mark.parametrize("T", [1, 17])
@pytest.mark.parametrize("exponent", [-20, -8])
def test_older_rows_of_a_negative_scale_keep_their_signs(exponent, T):
    c = Cache(1, 2, 64, 64, 128, BF, 64)
    k, v = (torch.ones(1, 2, T, 64, dtype=BF, device=DEV) for _ in range(2))
    for s in (c.ks, c.vs):
        s.fill_(-2.0 ** exponent)
    was = [c.rows(x, 0, 0, 40) for x in (c.k, c.v)]
    c.append(k, v, [40])
    for x, s, old in zip((c.k, c.v), (c.ks, c.vs), was):
        assert (c.factors(s, 0, 0, 1) == 2.0 ** -8).all()
        want, got = (-old * 2.0 ** (exponent + 8)).float().to(E4).double(), c.rows(x, 0, 0, 40)
        assert ((got == want) | (got.isnan() & want.isnan())).all()


@pytest.mark.parametrize("T", [1, 17])
@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf, -1.0])
def test_older_rows_without_a_scale_are_nan(bad, T):
    # no scale that the new rows can have gives them their values back
    c = Cache(1, 2, 128, 64, 128, FP, 64)
    k, v = (torch.ones(1, 2, T, 128, dtype=FP, device=DEV) for _ in range(2))
    for s in (c.ks, c.vs):
        s.fill_(bad)
    c.append(k, v, [40])
    for x, s in ((c.k, c.ks), (c.v, c.vs)):
        assert (c.factors(s, 0, 0, 1) == 2.0 ** -8).all()
        assert c.rows(x, 0, 0, 40).isnan().all()
        assert (c.rows(x, 0, 40, 40 + T) == 256.0).all()
