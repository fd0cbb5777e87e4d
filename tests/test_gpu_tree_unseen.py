"""Positions of a paged cache that no draft sees: whatever their rows hold, and
whatever page they are said to be on, they change nothing.  Masks need not be
trees: every draft may stand behind others, and a window hides drafts too."""
import math
import random

import pytest
import torch

import _mod_ref as R
from attention_forward_online_gb300 import osattn

pytestmark = pytest.mark.gpu
DEV, F64 = "cuda", torch.float64
BF, FP = torch.bfloat16, torch.float16


def visible(ctx, masks, window):
    """bool [T, ctx + T], by the definition in osattn.h."""
    T = len(masks)
    pos = [ctx + bin(m).count("1") - 1 for m in masks]
    at = list(range(ctx)) + pos
    see = torch.zeros(T, ctx + T, dtype=torch.bool)
    for t, m in enumerate(masks):
        for x in range(ctx + T):
            ok = m != 0 if x < ctx else bool((m >> (x - ctx)) & 1)
            see[t, x] = ok and (not window or abs(pos[t] - at[x]) < window)
    return see


def call(ctxs, masks, window, page, d, dtype, slopes=None, seed=0, H=4, Hkv=2, bad=-7):
    """Runs a batch whose unseen rows are NaN and whose pages without a visible
    key do not exist, and compares it with the 64-bit form."""
    B, T = len(ctxs), len(masks[0])
    g = torch.Generator(device=DEV).manual_seed(seed)
    per = -(-(max(ctxs) + T) // page)
    k, v = (torch.randn(B * per, Hkv, page, d, generator=g, device=DEV).to(dtype) for _ in range(2))
    order = torch.randperm(B * per, generator=torch.Generator().manual_seed(seed))
    table = order.to(torch.int32).reshape(B, per)
    given = torch.full_like(table, bad)
    for b in range(B):
        used = visible(ctxs[b], masks[b], window).any(0)
        for x in range(per * page):
            if x < ctxs[b] + T and bool(used[x]):
                given[b, x // page] = table[b, x // page]
        hidden = [x for x in range(per * page) if x >= ctxs[b] + T or not bool(used[x])]
        at = table[b, torch.tensor(hidden, dtype=torch.long) // page].long().to(DEV)
        for y in (k, v):
            y[at, :, torch.tensor(hidden, device=DEV) % page] = math.nan
    q = (torch.randn(B, T, H, d, generator=g, device=DEV) * 2).to(dtype).transpose(1, 2)
    mt = torch.tensor([[m - (1 << 64) if m >> 63 else m for m in row] for row in masks], dtype=torch.int64, device=DEV)
    o = torch.full_like(q, math.nan)
    lse = torch.full((B, H, T), math.nan, device=DEV)
    osattn.tree_attn(q, k, v, given.to(DEV), torch.tensor(ctxs, dtype=torch.int32, device=DEV), mt, slopes=slopes,
                     window=window, out=o, lse=lse)
    assert osattn.get_device_status() == osattn.OK
    want = R.tree_reference(q, k, v, table.to(DEV), ctxs, masks, 1 / math.sqrt(d), 0.0, slopes, window)
    R.check(o, *want["o"], "o")
    R.check(lse, *want["lse"], "lse")


TYPES = pytest.mark.parametrize("dtype,d", [(BF, 128), (FP, 64)], ids=["bf16-128", "fp16-64"])


@TYPES
@pytest.mark.parametrize("ctx", [100, 102, 103, 250])
def test_window_of_drafts_that_see_one_another(ctx, dtype, d):
    # both stand at ctx + 1: key ctx - window + 1 is hidden from them
    call([ctx], [[3, 3]], 8, 16, d, dtype)
    call([ctx, 9], [[15] * 4, [7] * 4], 20, 8, d, dtype)


@TYPES
def test_draft_that_only_the_window_hides(dtype, d):
    # draft 0 is on every line but its own, and a place or more away from all
    call([50], [[0, 3, 7, 15]], 1, 16, d, dtype)
    call([130], [[6, 2, 6, 13]], 1, 16, d, dtype)


@TYPES
@pytest.mark.parametrize("window", [0, 5])
def test_padding_needs_no_pages(window, dtype, d):
    # sequence 0: two drafts, six of padding that reach into the next page;
    # sequence 1: nothing but padding; sequence 2: a draft nobody sees
    call([14, 40, 30], [[1, 3] + [0] * 6, [0] * 8, [1, 0, 5, 9, 9, 9, 9, 9]], window, 16, d, dtype)


@TYPES
@pytest.mark.parametrize("seed", range(12))
def test_masks_of_any_kind(seed, dtype, d):
    rng = random.Random(seed)
    T = rng.choice([1, 2, 5, 17, 33, 64])
    window = rng.choice([0, 1, 2, 3, 7, 20, T, 100])
    B = 3
    ctxs = [rng.randrange(0, 400) for _ in range(B)]
    masks = []
    for b in range(B):
        few = rng.random() < 0.5
        row = []
        for t in range(T):
            m = rng.getrandbits(T) & (rng.getrandbits(T) if few else -1)
            row.append(m if m else 1 << rng.randrange(T))
        masks.append(row)
    masks[0] = [1 << rng.randrange(T) | 1 << rng.randrange(T)] * T
    slopes = torch.rand(4, generator=torch.Generator().manual_seed(seed)).to(DEV) if seed % 2 else None
    call(ctxs, masks, window, rng.choice([8, 16, 32]), d, dtype, slopes, seed)
