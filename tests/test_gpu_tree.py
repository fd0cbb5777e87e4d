"""GPU parity of tree attention over a paged cache (osattn_tree_attn) against
the 64-bit form of _mod_ref.py, every element within the bound derived there."""
import math
import random

import pytest
import torch

import _mod_ref as R
from attention_forward_online_gb300 import osattn

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF, FP = torch.bfloat16, torch.float16


def setup(B, H, Hkv, T, d, page, ctx, dtype, seed, extra=3, layout="phsd", trees=True, std=2.0):
    """Inputs with the pool in a random page order; rows of the cache that no
    sequence holds are NaN."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    rng = random.Random(seed)
    per = -(-(max(ctx) + T) // page) + 1
    pool = B * per + extra
    shape = (pool, Hkv, page, d) if layout == "phsd" else (pool, page, Hkv, d)
    k = torch.full(shape, math.nan, dtype=dtype, device=DEV)
    v = torch.full(shape, math.nan, dtype=dtype, device=DEV)
    if layout != "phsd":
        k, v = k.transpose(1, 2), v.transpose(1, 2)
    ids = list(range(pool))
    rng.shuffle(ids)
    table = torch.tensor(ids[:B * per], dtype=torch.int32).reshape(B, per).to(DEV)
    for b in range(B):
        n = ctx[b] + T
        keys = torch.arange(n, device=DEV)
        at = table[b].long()[keys // page]
        for x in (k, v):
            x[at, :, keys % page] = torch.randn(n, Hkv, d, generator=g, device=DEV).to(dtype)
    q = (torch.randn(B, T, H, d, generator=g, device=DEV) * std).to(dtype).transpose(1, 2)
    masks = []
    for b in range(B):
        m = []
        for u in range(T):
            parent = rng.randint(max(-1, u - 5), u - 1) if u else -1
            m.append((m[parent] if parent >= 0 else 0) | 1 << u)
        masks.append(m)
    if not trees:
        masks = [[(2 << t) - 1 for t in range(T)] for _ in range(B)]
    signed = [[m - (1 << 64) if m >> 63 else m for m in row] for row in masks]
    mt = torch.tensor(signed, dtype=torch.int64, device=DEV) if trees else None
    return q, k, v, table, torch.tensor(ctx, dtype=torch.int32, device=DEV), mt, masks


def run(q, k, v, table, ctx, mt, **kw):
    o = torch.full_like(q, math.nan)
    lse = torch.full(q.shape[:3], math.nan, dtype=torch.float32, device=DEV)
    osattn.tree_attn(q, k, v, table, ctx, mt, out=o, lse=lse, **kw)
    assert osattn.get_device_status() == osattn.OK
    return {"o": o, "lse": lse}


def compare(s, cap=0.0, slopes=None, window=0, scale=None):
    q, k, v, table, ctx, mt, masks = s
    sc = 1 / math.sqrt(q.shape[3]) if scale is None else scale
    got = run(q, k, v, table, ctx, mt, softcap=cap, slopes=slopes, window=window, scale=scale)
    want = R.tree_reference(q, k, v, table, ctx.tolist(), masks, sc, cap, slopes, window)
    for n, (val, bound) in want.items():
        R.check(got[n], val, bound, n)
    return got


def slopes_of(H):
    return torch.exp2(-8.0 * torch.arange(1, H + 1, device=DEV, dtype=torch.float32) / H)


# B, H, Hkv, T, page, ctx
SHAPES = [
    (1, 1, 1, 1, 8, [0]),
    (1, 4, 1, 1, 16, [127]),
    (2, 4, 4, 1, 16, [128, 1]),
    (3, 6, 2, 1, 32, [0, 5000, 77]),
    (1, 8, 2, 7, 64, [250]),
    (5, 8, 1, 13, 128, [0, 121, 122, 1000, 300]),
    (2, 10, 2, 27, 256, [3000, 100]),
    (2, 8, 1, 64, 16, [64, 1500]),
    (1, 16, 1, 64, 384, [700]),
    (40, 4, 2, 3, 16, [(37 * x) % 600 for x in range(40)]),
    (1, 96, 1, 3, 16, [200]),    # one token a row tile
    (2, 128, 1, 2, 8, [130, 9]),  # a group that fills the tile
    (1, 8, 1, 2, 64, [9000]),    # many partials a row
    (1, 20, 1, 9, 16, [20011]),
    (700, 1, 1, 1, 8, [x % 20 for x in range(700)]),  # more sequences than threads
]


@pytest.mark.parametrize("dtype,d", [(BF, 128), (FP, 64), (BF, 64), (FP, 128)],
                         ids=["bf16-128", "fp16-64", "bf16-64", "fp16-128"])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: f"B{s[0]}H{s[1]}k{s[2]}T{s[3]}p{s[4]}")
def test_shapes(shape, dtype, d):
    B, H, Hkv, T, page, ctx = shape
    compare(setup(B, H, Hkv, T, d, page, ctx, dtype, seed=T + d))


@pytest.mark.parametrize("T", [1, 33])
@pytest.mark.parametrize("kind", ["cap", "slopes", "both"])
@pytest.mark.parametrize("window", [0, 1, 20, 200])
def test_scores_and_windows(kind, window, T):
    a = {}
    if kind != "slopes":
        a["cap"] = 4.0
    if kind != "cap":
        a["slopes"] = slopes_of(8)
    compare(setup(3, 8, 2, T, 64, 32, [500, 130, 3], BF, seed=7), window=window, **a)


def test_no_mask_is_a_chain_and_other_layouts():
    compare(setup(2, 8, 2, 20, 128, 16, [333, 90], BF, seed=1, layout="pshd", trees=False))
    compare(setup(2, 8, 2, 64, 64, 64, [200, 10], FP, seed=2, layout="pshd", trees=False), window=30)


@pytest.mark.parametrize("scale", [-0.3, 0.0])
def test_scales(scale):
    compare(setup(1, 4, 2, 5, 64, 16, [400], BF, seed=3), scale=scale)


def test_padding_drafts_see_nothing_and_may_hold_anything():
    q, k, v, table, ctx, mt, masks = setup(3, 8, 2, 9, 64, 16, [120, 40, 300], BF, seed=4)
    for b, n in ((0, 5), (1, 0), (2, 1)):  # drafts from n on are padding
        for u in range(n, 9):
            masks[b][u] = 0
            mt[b, u] = 0
            q[b, :, u] = math.nan
            key = int(ctx[b]) + u
            for x in (k, v):
                x[int(table[b, key // 16]), :, key % 16] = math.nan
    got = compare((q.nan_to_num(0.0), k, v, table, ctx, mt, masks))
    dirty = run(q, k, v, table, ctx, mt)
    for n in got:
        assert torch.equal(got[n], dirty[n]), n
    assert (dirty["o"][1] == 0).all() and (dirty["lse"][1] == -math.inf).all()


def test_masks_that_are_no_tree():
    q, k, v, table, ctx, mt, masks = setup(2, 4, 2, 64, 64, 16, [70, 200], FP, seed=5)
    rng = random.Random(5)
    for b in range(2):
        for t in range(64):
            masks[b][t] = rng.getrandbits(64) | 1 << rng.randrange(64)
            m = masks[b][t]
            mt[b, t] = m - (1 << 64) if m >> 63 else m
    compare((q, k, v, table, ctx, mt, masks), slopes=slopes_of(4), window=50)


def test_bits_behind_the_drafts_say_nothing():
    q, k, v, table, ctx, mt, masks = setup(1, 4, 2, 6, 64, 16, [70], BF, seed=6)
    clean = run(q, k, v, table, ctx, mt)
    dirty = run(q, k, v, table, ctx, mt | (-1 << 6))
    for n in clean:
        assert torch.equal(clean[n], dirty[n])


def test_pages_before_the_window_need_not_exist():
    q, k, v, table, ctx, mt, masks = setup(2, 4, 2, 4, 128, 16, [1000, 300], BF, seed=8)
    want = run(q, k, v, table, ctx, mt, window=100)
    for b, n in ((0, 1000), (1, 300)):
        gone = (n - 100 + 1) // 16  # pages wholly before the first visible key
        k[table[b, :gone].long()] = math.nan
        table[b, :gone] = -7
    got = run(q, k, v, table, ctx, mt, window=100)
    for n in want:
        assert torch.equal(want[n], got[n]), n


def test_a_bad_page_is_reported_and_reads_as_zeros():
    q, k, v, table, ctx, mt, masks = setup(2, 4, 2, 2, 64, 16, [100, 50], BF, seed=9)
    zeroed = table.clone()
    k2, v2 = k.clone(), v.clone()
    k2[table[0, 2].long()] = 0
    v2[table[0, 2].long()] = 0
    want = run(q, k2, v2, zeroed, ctx, mt)
    for bad in (-1, k.shape[0], 2 ** 31 - 1, -2 ** 31):
        table[0, 2] = bad
        o, lse = osattn.tree_attn(q, k, v, table, ctx, mt)
        assert osattn.get_device_status() == osattn.ERR_INVALID_ARG
        assert torch.equal(o, want["o"]) and torch.equal(lse, want["lse"])


def test_context_lengths_outside_the_table_are_clamped_and_reported():
    q, k, v, table, ctx, mt, masks = setup(2, 4, 2, 2, 64, 16, [100, 50], BF, seed=10)
    k, v = k.nan_to_num(0.5), v.nan_to_num(0.5)
    most = table.shape[1] * 16 - 2
    good = run(q, k, v, table, torch.tensor([most, 0], dtype=torch.int32, device=DEV), mt)
    o, lse = osattn.tree_attn(q, k, v, table, torch.tensor([most + 9, -4], dtype=torch.int32, device=DEV), mt)
    assert osattn.get_device_status() == osattn.ERR_INVALID_ARG
    assert torch.equal(o, good["o"]) and torch.equal(lse, good["lse"])


def test_long_cache_with_far_pages():
    # element offsets beyond 2^31: 40000 pages of 8 x 128 x 64 values
    B, H, Hkv, T, d, page = 1, 8, 8, 3, 64, 128
    pool = 40000
    k = torch.zeros(pool, Hkv, page, d, dtype=BF, device=DEV)
    v = torch.zeros_like(k)
    g = torch.Generator(device=DEV).manual_seed(12)
    ids = [39999, 5, 33000, 39000]
    for i in ids:
        k[i] = torch.randn(Hkv, page, d, generator=g, device=DEV).to(BF)
        v[i] = torch.randn(Hkv, page, d, generator=g, device=DEV).to(BF)
    table = torch.tensor([ids], dtype=torch.int32, device=DEV)
    q = torch.randn(B, H, T, d, generator=g, device=DEV).to(BF)
    ctx = torch.tensor([400], dtype=torch.int32, device=DEV)
    masks = [[1, 3, 5]]
    compare((q, k, v, table, ctx, torch.tensor(masks, dtype=torch.int64, device=DEV), masks))


def test_same_bits_again_in_a_graph_and_with_one_workspace():
    s1 = setup(4, 8, 2, 5, 128, 16, [900, 30, 400, 128], BF, seed=11)
    s2 = setup(2, 4, 1, 1, 128, 16, [2000, 3], BF, seed=12)
    want = [run(*s[:6]) for s in (s1, s2)]
    for s, w in zip((s1, s2), want):
        again = run(*s[:6])
        for n in w:
            assert torch.equal(w[n], again[n]), n
    need = max(osattn.tree_workspace_bytes(s[0].shape[0], s[0].shape[1], s[1].shape[1], s[0].shape[2], 128)
               for s in (s1, s2))
    ws = torch.full((need,), 0xff, dtype=torch.uint8, device=DEV)  # NaN everywhere
    graphs, outs = [], []
    for s in (s1, s2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(osattn.tree_attn(*s[:6], workspace=ws))
        graphs.append(graph)
    for _ in range(2):
        for x in outs:
            x[0].fill_(math.nan)
        for graph in graphs:
            graph.replay()
    torch.cuda.synchronize()
    for (o, lse), w in zip(outs, want):
        assert torch.equal(o, w["o"]) and torch.equal(lse, w["lse"])
    # the context grows between replays: lengths are read when the graph runs
    # (bits compared: the key after the last draft's, now seen, was left NaN)
    s1[4].add_(1)
    graphs[0].replay()
    grown = run(*s1[:6])
    assert torch.equal(outs[0][0].view(torch.int16), grown["o"].view(torch.int16))
    assert not torch.equal(outs[0][0].view(torch.int16), want[0]["o"].view(torch.int16))


def test_two_streams_at_once():
    sets = [setup(2, 8, 2, 5, 64, 16, [900, 300], BF, seed=20 + s) for s in (0, 1)]
    want = [run(*s[:6]) for s in sets]
    streams = [torch.cuda.Stream() for _ in sets]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    for _ in range(5):
        got = [osattn.tree_attn(*s[:6], stream=st) for s, st in zip(sets, streams)]
    torch.cuda.synchronize()
    for (o, lse), w in zip(got, want):
        assert torch.equal(o, w["o"]) and torch.equal(lse, w["lse"])


def test_decode_continues_what_the_prompt_pass_computed():
    # a prompt's rows by fwd_mod, then the same rows as drafts over the cache
    B, H, Hkv, N, T, d, page = 2, 8, 2, 300, 6, 128, 32
    g = torch.Generator(device=DEV).manual_seed(30)
    q = (torch.randn(B, H, N, d, generator=g, device=DEV) * 2).to(BF)
    k = torch.randn(B, Hkv, N, d, generator=g, device=DEV).to(BF)
    v = torch.randn(B, Hkv, N, d, generator=g, device=DEV).to(BF)
    slopes = slopes_of(H)
    o, lse = osattn.fwd_mod(q, k, v, plan=osattn.mask_plan(B, N, N, causal=True, window=150, device=DEV),
                            softcap=6.0, slopes=slopes)
    per = -(-N // page)
    pad = per * page - N
    pages = [torch.nn.functional.pad(x, (0, 0, 0, pad)).reshape(B, Hkv, per, page, d).transpose(1, 2)
             .reshape(B * per, Hkv, page, d).contiguous() for x in (k, v)]
    table = torch.arange(B * per, dtype=torch.int32, device=DEV).reshape(B, per)
    ctx = torch.full((B,), N - T, dtype=torch.int32, device=DEV)
    o2, lse2 = osattn.tree_attn(q[:, :, N - T:], *pages, table, ctx, softcap=6.0, slopes=slopes, window=150)
    masks = [[(2 << t) - 1 for t in range(T)]] * B
    want = R.tree_reference(q[:, :, N - T:], *pages, table, ctx.tolist(), masks, d ** -0.5, 6.0, slopes, 150)
    for got in ((o[:, :, N - T:], lse[:, :, N - T:]), (o2, lse2)):
        R.check(got[0], *want["o"], "o")
        R.check(got[1], *want["lse"], "lse")
