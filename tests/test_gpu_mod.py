"""GPU parity of modified-score attention (osattn_mask_plan, osattn_fwd_mod,
osattn_bwd_mod) against the 64-bit forms of _mod_ref.py, every output element
within the bound derived there."""
import math
import os
import subprocess
import sys

import pytest
import torch

import _mod_ref as R
from attention_forward_online_gb300 import osattn

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF, FP = torch.bfloat16, torch.float16


def tensors(B, H, Hkv, Nq, Nkv, d, dtype, seed, bnhd=False, std=2.0):
    g = torch.Generator(device=DEV).manual_seed(seed)

    def mk(h, n, s):
        shape = (B, n, h, d) if bnhd else (B, h, n, d)
        t = (torch.randn(*shape, generator=g, device=DEV) * s).to(dtype)
        return t.transpose(1, 2) if bnhd else t

    return mk(H, Nq, std), mk(Hkv, Nkv, 1.0), mk(Hkv, Nkv, 1.0), mk(H, Nq, 1.0)


def slopes_of(H):
    return torch.exp2(-8.0 * torch.arange(1, H + 1, device=DEV, dtype=torch.float32) / H)


def i32(x):
    return None if x is None else torch.tensor(x, dtype=torch.int32, device=DEV)


def run(q, k, v, do, masks, cap=0.0, slopes=None, table=None, rel_map=None, plan=True, scale=None, nan=True):
    """The library's outputs into NaN-filled buffers."""
    B, Nq, Nkv = q.shape[0], q.shape[2], k.shape[2]
    p = osattn.mask_plan(B, Nq, Nkv, **masks, device=DEV) if plan else None
    mods = dict(scale=scale, plan=p, softcap=cap, slopes=slopes, rel_table=table, rel_map=rel_map)
    o = torch.full_like(q, math.nan)
    lse = torch.full(q.shape[:3], math.nan, dtype=torch.float32, device=DEV)
    osattn.fwd_mod(q, k, v, out=o, lse=lse, **mods)
    got = {"o": o, "lse": lse}
    grads = [torch.full_like(x, math.nan) for x in (q, k, v)]
    drel = None if table is None else torch.full_like(table, math.nan)
    osattn.bwd_mod(q, k, v, o, lse, do, dq=grads[0], dk=grads[1], dv=grads[2], drel=drel, **mods)
    got.update(zip(("dq", "dk", "dv"), grads))
    if drel is not None:
        got["drel"] = drel
    assert osattn.get_device_status() == osattn.OK
    return got


def compare(q, k, v, do, masks, cap=0.0, slopes=None, table=None, rel_map=None, plan=True, scale=None):
    B, Nq, Nkv = q.shape[0], q.shape[2], k.shape[2]
    sc = 1 / math.sqrt(q.shape[3]) if scale is None else scale
    see = R.visible(B, Nq, Nkv, **masks, device=DEV) if plan else R.visible(B, Nq, Nkv, device=DEV)
    got = run(q, k, v, do, masks, cap, slopes, table, rel_map, plan, scale)
    want = R.reference(q, k, v, see, sc, do, cap, slopes, table, rel_map, masks.get("q_offset", 0))
    for n, (val, bound) in want.items():
        R.check(got[n], val, bound, n)
    return got


# B, H, Hkv, Nq, Nkv, masks
MASKS = [
    (1, 1, 1, 1, 1, {}),
    (2, 2, 1, 1, 300, dict(causal=True, q_offset=299)),
    (1, 4, 2, 129, 129, dict(causal=True)),
    (2, 3, 3, 257, 400, dict(causal=True, q_offset=143)),
    (2, 4, 1, 300, 300, dict(causal=True, key_len=[300, 0])),
    (3, 2, 2, 200, 333, dict(key_len=[1, 128, 333])),
    (2, 4, 2, 385, 385, dict(causal=True, window=50)),
    (1, 2, 1, 600, 600, dict(window=130)),
    (2, 2, 1, 290, 290, dict(causal=True, prefix_len=[129, 17])),
    (1, 2, 2, 520, 520, dict(causal=True, window=40, prefix_len=[300])),
    (1, 2, 1, 140, 260, dict(causal=True, q_offset=-20)),
    (1, 2, 1, 300, 200, dict(causal=True, window=64, q_offset=50)),
]


@pytest.mark.parametrize("dtype,d", [(BF, 128), (FP, 64)], ids=["bf16-128", "fp16-64"])
@pytest.mark.parametrize("case", MASKS, ids=lambda c: "x".join(map(str, c[:5])) + "-" + "-".join(c[5]))
def test_masks(case, dtype, d):
    B, H, Hkv, Nq, Nkv, masks = case
    masks = {n: i32(x) if isinstance(x, list) else x for n, x in masks.items()}
    compare(*tensors(B, H, Hkv, Nq, Nkv, d, dtype, seed=Nq + d), masks)


def documents(kind, B, N):
    g = torch.Generator().manual_seed(N)
    if kind == "short":
        return (torch.rand(B, N, generator=g) < 0.05).long().cumsum(1).int()
    if kind == "ones":
        return torch.arange(N).repeat(B, 1).int()
    if kind == "single":
        return torch.full((B, N), 7, dtype=torch.int32)
    if kind == "padded":  # documents, then padding that sees nothing; one row all padding
        ids = (torch.rand(B, N, generator=g) < 0.02).long().cumsum(1).int()
        ids[0, N // 3:] = -1
        ids[-1] = -5
        return ids
    return torch.randint(-1, 2, (B, N), generator=g, dtype=torch.int32)  # ids that come again, runs of one


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("kind", ["short", "ones", "single", "padded", "again"])
def test_documents(kind, causal):
    ids = documents(kind, 2, 450).to(DEV)
    compare(*tensors(2, 2, 1, 450, 450, 64, BF, seed=5), dict(causal=causal, doc_ids=ids))
    # queries that are a part of the keys
    compare(*tensors(2, 2, 2, 150, 450, 128, BF, seed=6), dict(causal=causal, doc_ids=ids, q_offset=217))


def test_long_documents_cross_many_tiles():
    N = 9001
    ids = torch.zeros(1, N, dtype=torch.int32, device=DEV)
    ids[0, 40:] = 1
    ids[0, 8900:] = 2
    plan = osattn.mask_plan(1, N, N, doc_ids=ids)
    tiles = -(-N // 128)
    rows = plan.buffer[tiles * 16:].view(torch.int32).reshape(N, 2)
    edge = torch.tensor([0, 40, 8900, N], device=DEV)
    assert torch.equal(rows[:, 0].long(), edge[ids[0].long()])
    assert torch.equal(rows[:, 1].long(), edge[ids[0].long() + 1])


SCORES = ["cap", "slopes", "cap_slopes", "rel", "rel_one_sided", "rel_wide", "rel_holes"]


def score_args(kind, H, dtype):
    g = torch.Generator(device=DEV).manual_seed(11)
    a = {}
    if kind.startswith("cap"):
        a["cap"] = 5.0
    if kind.endswith("slopes"):
        a["slopes"] = slopes_of(H)
    if kind.startswith("rel"):
        nb = 32
        m = osattn.rel_buckets(nb, 1024 if kind == "rel_wide" else 40, kind != "rel_one_sided")
        if kind == "rel_holes":
            m[::7] = -1
            m[3::11] = nb + 3
        a["rel_map"] = m.to(DEV)
        a["table"] = torch.randn(nb, H, generator=g, device=DEV).to(dtype)
    return a


@pytest.mark.parametrize("dtype,d", [(BF, 64), (BF, 128), (FP, 64), (FP, 128)],
                         ids=["bf16-64", "bf16-128", "fp16-64", "fp16-128"])
@pytest.mark.parametrize("kind", SCORES)
def test_scores(kind, dtype, d):
    q, k, v, do = tensors(2, 4, 2, 500, 500, d, dtype, seed=21, bnhd=True)
    compare(q, k, v, do, dict(key_len=i32([500, 333])), **score_args(kind, 4, dtype))
    q, k, v, do = tensors(1, 2, 2, 200, 410, d, dtype, seed=22)
    compare(q, k, v, do, dict(causal=True, q_offset=210), **score_args(kind, 2, dtype))


@pytest.mark.parametrize("kind", ["cap", "slopes", "rel"])
def test_no_plan_and_one_token(kind):
    compare(*tensors(2, 2, 1, 1, 1, 64, BF, seed=3), {}, plan=False, **score_args(kind, 2, BF))
    compare(*tensors(1, 2, 1, 131, 259, 128, BF, seed=4), {}, plan=False, **score_args(kind, 2, BF))


@pytest.mark.parametrize("scale", [-0.2, 0.0, 1.0])
@pytest.mark.parametrize("kind", ["plain", "cap", "slopes", "rel"])
def test_scales(kind, scale):
    a = {} if kind == "plain" else score_args(kind, 2, BF)
    compare(*tensors(1, 2, 1, 150, 280, 64, BF, seed=8), dict(key_len=i32([270])), scale=scale, **a)


def test_scores_far_beyond_the_cap():
    # raw scores of some hundreds against a cap of 2: every tanh is saturated
    compare(*tensors(1, 2, 2, 140, 140, 64, BF, seed=9, std=60.0), dict(causal=True), cap=2.0)


@pytest.mark.parametrize("cap", [1e-3, 0.5, 300.0, 1e4])
def test_caps_of_every_size(cap):
    compare(*tensors(1, 2, 1, 150, 200, 64, BF, seed=10), dict(key_len=i32([190])), cap=cap)
    # scores on both sides of 0.4 cap, where the form of the tanh changes
    compare(*tensors(1, 2, 1, 150, 200, 64, FP, seed=13, std=cap if 0.1 < cap < 1e3 else 2.0), {}, cap=cap)


# few key tiles: their queries are shared out to 8, 4, 2 CTAs; the last one's
# windows leave some of them nothing
SHARED = [
    (1, 8, 1, 600, 900, dict(causal=True, q_offset=300, key_len=[777])),
    (2, 4, 2, 500, 700, dict(key_len=[700, 130])),
    (3, 4, 2, 400, 1000, dict(causal=True, q_offset=600)),
    (1, 2, 1, 1500, 1500, dict(causal=True, window=4)),
]


@pytest.mark.parametrize("kind", ["plain", "cap", "slopes", "rel"])
@pytest.mark.parametrize("dtype,d", [(BF, 128), (FP, 64)], ids=["bf16-128", "fp16-64"])
@pytest.mark.parametrize("case", SHARED, ids=lambda c: "x".join(map(str, c[:5])))
def test_key_tiles_shared_by_ctas(case, dtype, d, kind):
    B, H, Hkv, Nq, Nkv, masks = case
    masks = {k: i32(v) if isinstance(v, list) else v for k, v in masks.items()}
    compare(*tensors(B, H, Hkv, Nq, Nkv, d, dtype, seed=21, bnhd=True), masks, **score_args(kind, H, dtype))


@pytest.mark.parametrize("fill", [math.nan, math.inf, -math.inf, 3e38])
@pytest.mark.parametrize("kind", ["plain", "cap", "slopes", "rel"])
def test_masked_places_hold_anything(kind, fill):
    # behind each sequence's last key, and in queries that see nothing
    B, H, N, d = 2, 2, 300, 128
    q, k, v, do = tensors(B, H, 1, N, N, d, BF, seed=31)
    ids = torch.zeros(B, N, dtype=torch.int32, device=DEV)
    ids[0, 170:] = -1
    ids[1, 40:] = -1
    masks = dict(causal=True, doc_ids=ids)
    a = {} if kind == "plain" else score_args(kind, H, BF)
    clean = run(q, k, v, do, masks, **a)
    for b, n in ((0, 170), (1, 40)):
        for x in (q, k, v, do):
            x[b, :, n:] = fill
    dirty = run(q, k, v, do, masks, **a)
    for n in clean:
        assert torch.equal(clean[n], dirty[n]), n
    for b, n in ((0, 170), (1, 40)):
        assert (dirty["o"][b, :, n:] == 0).all() and (dirty["lse"][b, :, n:] == -math.inf).all()
        for g in ("dq", "dk", "dv"):
            assert (dirty[g][b, :, n:] == 0).all()


@pytest.mark.parametrize("dtype,d", [(BF, 128), (FP, 64)], ids=["bf16-128", "fp16-64"])
def test_bias_gradients_sum_to_zero(dtype, d):
    # A row's dY sum to 0, so a head's table gradients do, but for the rounding
    # of each to 16 bits (half a step) and what P, with its exponent and LSE in
    # fp32, is off (2^-20) times the greatest |dY| there can be, 2 |dO| |V|.
    q, k, v, do = tensors(2, 4, 2, 300, 333, d, dtype, seed=41)
    got = run(q, k, v, do, {}, **score_args("rel", 4, dtype))
    drel = got["drel"].double()
    most = 2 * do.double().norm(dim=-1).max() * v.double().norm(dim=-1).max()
    bound = drel.abs().sum(0) * torch.finfo(dtype).eps / 2 + 2 * 300 * most * 2.0**-20
    assert (drel.sum(0).abs() <= bound).all(), (drel.sum(0), bound)


@pytest.mark.parametrize("kind", ["plain", "cap", "slopes", "rel"])
def test_large_values(kind):
    q, k, v, do = tensors(1, 2, 1, 200, 300, 64, BF, seed=31)
    args = score_args(kind, 2, BF)
    if kind == "rel":
        args["table"] = args["table"] * 3  # biases some 20 apart
    compare(q, k, v * 2.0**50, do * 2.0**-60, {}, **args)


def test_key_tails_hold_anything():
    # keys behind key_len, with queries everywhere
    q, k, v, do = tensors(2, 2, 2, 200, 300, 64, BF, seed=32)
    masks = dict(key_len=i32([130, 255]))
    clean = run(q, k, v, do, masks)
    for b, n in ((0, 130), (1, 255)):
        k[b, :, n:] = math.nan
        v[b, :, n:] = math.inf
    dirty = run(q, k, v, do, masks)
    for n in clean:
        assert torch.equal(clean[n], dirty[n]), n


def test_same_bits_again_and_in_a_graph():
    q, k, v, do = tensors(2, 4, 2, 700, 700, 64, BF, seed=41)
    a = score_args("rel", 4, BF)
    masks = dict(causal=True, window=200)
    first = run(q, k, v, do, masks, **a)
    again = run(q, k, v, do, masks, **a)
    for n in first:
        assert torch.equal(first[n], again[n]), n

    def step():
        plan = osattn.mask_plan(2, 700, 700, **masks, device=DEV)
        mods = dict(plan=plan, rel_table=a["table"], rel_map=a["rel_map"])
        o, lse = osattn.fwd_mod(q, k, v, **mods)
        return (o, lse, *osattn.bwd_mod(q, k, v, o, lse, do, **mods))

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = step()
    for _ in range(2):
        for x in outs:
            x.fill_(math.nan)
        graph.replay()
        torch.cuda.synchronize()
        for x, n in zip(outs, ("o", "lse", "dq", "dk", "dv", "drel")):
            assert torch.equal(x, first[n]), n


def test_first_call_of_a_process_may_be_captured():
    code = """
import torch
from attention_forward_online_gb300 import osattn
g = torch.Generator(device="cuda").manual_seed(1)
q, k, v = (torch.randn(1, 2, 200, 64, generator=g, device="cuda").to(torch.bfloat16) for _ in range(3))
osattn.fwd(q, k, v)  # the library's set-up of the device
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    plan = osattn.mask_plan(1, 200, 200, causal=True, device="cuda")
    o, lse = osattn.fwd_mod(q, k, v, plan=plan, softcap=5.0)
    grads = osattn.bwd_mod(q, k, v, o, lse, q, plan=plan, softcap=5.0)
graph.replay()
torch.cuda.synchronize()
plan = osattn.mask_plan(1, 200, 200, causal=True, device="cuda")
o2, lse2 = osattn.fwd_mod(q, k, v, plan=plan, softcap=5.0)
assert torch.equal(o, o2) and torch.equal(lse, lse2)
for a, b in zip(grads, osattn.bwd_mod(q, k, v, o, lse, q, plan=plan, softcap=5.0)):
    assert torch.equal(a, b)
assert osattn.get_device_status() == 0
"""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    subprocess.run([sys.executable, "-c", code], check=True, cwd=root, timeout=120)


def test_two_streams_at_once():
    sets = [(tensors(2, 2, 1, 600, 600, 64, BF, seed=s), dict(causal=True, window=100 * s)) for s in (1, 2)]
    alone = [run(*t, m) for t, m in sets]
    streams = [torch.cuda.Stream() for _ in sets]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    got = []
    for _ in range(3):
        got = []
        for (t, m), s in zip(sets, streams):
            q, k, v, do = t
            plan = osattn.mask_plan(2, 600, 600, **m, device=DEV, stream=s)
            o, lse = osattn.fwd_mod(q, k, v, plan=plan, stream=s)
            got.append((o, lse, *osattn.bwd_mod(q, k, v, o, lse, do, plan=plan, stream=s)))
    torch.cuda.synchronize()
    for a, g in zip(alone, got):
        for x, n in zip(g, ("o", "lse", "dq", "dk", "dv")):
            assert torch.equal(x, a[n]), n


def test_a_plan_for_other_sizes_is_refused():
    q, k, v, _ = tensors(1, 2, 2, 64, 64, 64, BF, seed=1)
    with pytest.raises(ValueError):
        osattn.fwd_mod(q, k, v, plan=osattn.mask_plan(1, 64, 65, causal=True))
    with pytest.raises(osattn.OsattnError):
        osattn.fwd_mod(q.float(), k.float(), v.float())
    with pytest.raises(osattn.OsattnError):
        osattn.fwd_mod(q, k, v, softcap=2.0, **{n: x for n, x in
                                                zip(("rel_table", "rel_map"),
                                                    (torch.zeros(4, 2, dtype=BF, device=DEV), i32([0, 1, 2])))})
