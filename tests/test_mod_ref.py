"""CPU checks of the 64-bit forms that the modified-score GPU tests compare
with: gradients against central differences and the written-out formula, the
masks against a loop over pairs, the bucket map, and the refusals of the
entry points (which need no GPU)."""
import ctypes
import math

import pytest
import torch

import _mod_ref as R
from attention_forward_online_gb300 import osattn

P = 0x10000  # an aligned address; validation fails before it is used


def small(seed=0, H=2, Hkv=1, Nq=5, Nkv=6, d=4):
    g = torch.Generator().manual_seed(seed)
    mk = lambda h, n: torch.randn(1, h, n, d, generator=g, dtype=torch.float64)  # noqa: E731
    return mk(H, Nq), mk(Hkv, Nkv), mk(Hkv, Nkv), mk(H, Nq), g


@pytest.mark.parametrize("cap,slope,rel", [(0, 0, 0), (1.5, 0, 0), (0, 1, 0), (1.5, 1, 0), (0, 0, 1)])
def test_reference_gradients_match_differences_and_formula(cap, slope, rel):
    q, k, v, do, g = small()
    see = R.visible(1, 5, 6, causal=True, q_offset=1)
    see[0, 3] = False
    slopes = torch.tensor([0.3, 0.1], dtype=torch.float64) if slope else None
    table = torch.randn(3, 2, generator=g, dtype=torch.float64) if rel else None
    rel_map = torch.tensor([2, 0, 1, 5, 2], dtype=torch.int32) if rel else None

    def f(q, k, v, table):
        y = R.logits(q, k.repeat_interleave(2, 1), 0.5, cap, slopes, table, rel_map, 1)
        return (R.softmax_out(y, see[:, None], v.repeat_interleave(2, 1))[0] * do).sum()

    leaves = [x.clone().requires_grad_() for x in (q, k, v)] + ([table.clone().requires_grad_()] if rel else [])
    got = torch.autograd.grad(f(*leaves[:3], leaves[3] if rel else None), leaves)
    for n, x in enumerate(leaves):
        flat = x.detach().reshape(-1)
        for i in range(flat.numel()):
            vals = []
            for h in (1e-5, -1e-5):
                moved = [y.detach().clone() for y in leaves]
                moved[n].reshape(-1)[i] += h
                vals.append(float(f(*moved[:3], moved[3] if rel else None)))
            # central differences err by h^2 times a third derivative of order 10
            assert abs((vals[0] - vals[1]) / 2e-5 - float(got[n].reshape(-1)[i])) < 1e-7
    # dQ from the formula
    y = R.logits(q, k.repeat_interleave(2, 1), 0.5, cap, slopes, table, rel_map, 1)
    vv = v.repeat_interleave(2, 1)
    o, _, p = R.softmax_out(y, see[:, None], vv)
    ds = p * (do @ vv.transpose(-1, -2) - (do * o).sum(-1, keepdim=True))
    if cap:
        raw = 0.5 * (q @ k.repeat_interleave(2, 1).transpose(-1, -2))
        ds = ds * (1 - torch.tanh(raw / cap) ** 2)
    assert torch.allclose(0.5 * ds @ k.repeat_interleave(2, 1), got[0], atol=1e-12)


@pytest.mark.parametrize("off", [0, 3, -2])
def test_visible_matches_a_loop_over_pairs(off):
    B, Nq, Nkv = 3, 9, 11
    ids = torch.tensor([[0, 0, 0, 1, 1, 2, 2, 2, 0, 0, 0], [4] * 11,
                        [-1, 0, 0, -1, -1, 3, 3, 3, 3, -2, -2]], dtype=torch.int32)
    kl, pf = [11, 7, 0], [2, 0, 5]
    got = R.visible(B, Nq, Nkv, True, 4, off, kl, pf, ids)
    for b in range(B):
        for i in range(Nq):
            p = i + off
            for j in range(Nkv):
                ok = j < kl[b] and (j <= p or j < pf[b]) and abs(j - p) < 4 and 0 <= p < Nkv
                if ok:
                    lo, hi = min(j, p), max(j, p)
                    ok = ids[b, p] >= 0 and all(int(ids[b, x]) == int(ids[b, p]) for x in range(lo, hi + 1))
                assert bool(got[b, i, j]) == ok, (b, i, j)


def test_rel_buckets_sides_and_order():
    m = osattn.rel_buckets(32, 128)
    assert m.dtype == torch.int32 and m.numel() == 257
    assert int(m[128]) == 0 and int(m[0]) == 15 and int(m[256]) == 31 and int(m[127]) == 1 and int(m[129]) == 17
    left = m[:129].flip(0)
    assert (left[1:] >= left[:-1]).all() and int(m.max()) == 31
    one = osattn.rel_buckets(32, 128, bidirectional=False)
    assert (one[128:] == 0).all() and int(one[0]) == 31
    with pytest.raises(ValueError):
        osattn.rel_buckets(2, 128)


@pytest.fixture(scope="module")
def L():
    from attention_forward_online_gb300 import _build

    _build.build()
    return osattn.lib()


def fwd(**kw):
    a = dict(q=P, k=P, v=P, o=P, lse=P, B=1, H=4, Hkv=2, Nq=8, Nkv=8, d=64, strides=(None,) * 4,
             scale=0.125, score=osattn._Score(), plan=None, dtype=osattn.BF16)
    a.update(kw)
    st = [None if s is None else (ctypes.c_int64 * 3)(*s) for s in a["strides"]]
    return osattn.lib().osattn_fwd_mod(a["q"], a["k"], a["v"], a["o"], a["lse"], a["B"], a["H"], a["Hkv"],
                                       a["Nq"], a["Nkv"], a["d"], *st, a["scale"],
                                       None if a["score"] is None else ctypes.byref(a["score"]), a["plan"],
                                       a["dtype"], None)


def bwd(**kw):
    a = dict(p=[P] * 9, drel=None, B=1, H=4, Hkv=2, Nq=8, Nkv=8, d=64, strides=(None,) * 8, scale=0.125,
             score=osattn._Score(), plan=None, dtype=osattn.BF16, ws=P, ws_bytes=1 << 20)
    a.update(kw)
    st = [None if s is None else (ctypes.c_int64 * 3)(*s) for s in a["strides"]]
    return osattn.lib().osattn_bwd_mod(*a["p"], a["drel"], a["B"], a["H"], a["Hkv"], a["Nq"], a["Nkv"],
                                       a["d"], *st, a["scale"], ctypes.byref(a["score"]), a["plan"],
                                       a["dtype"], a["ws"], a["ws_bytes"], None)


def rel_score(**kw):
    a = dict(rel_table=P, rel_map=P, rel_num=8, rel_range=16)
    a.update(kw)
    return osattn._Score(**a)


BAD, NOT = osattn.ERR_INVALID_ARG, osattn.ERR_UNSUPPORTED


@pytest.mark.parametrize("kw,expect", [
    (dict(q=None), BAD), (dict(lse=None), BAD), (dict(k=P + 8), BAD), (dict(Hkv=3), BAD), (dict(Hkv=0), BAD),
    (dict(Nq=0), BAD), (dict(Nkv=0), BAD), (dict(B=0), BAD), (dict(plan=P + 8), BAD),
    (dict(Nq=(1 << 30) + 1), BAD), (dict(scale=math.inf), BAD), (dict(d=80), NOT), (dict(dtype=osattn.FP32), NOT),
    (dict(score=osattn._Score(softcap=-1.0)), BAD), (dict(score=osattn._Score(softcap=math.nan)), BAD),
    (dict(score=osattn._Score(softcap=math.inf)), BAD), (dict(score=osattn._Score(softcap=9e-4)), BAD),
    (dict(score=osattn._Score(softcap=10001.0)), BAD), (dict(score=osattn._Score(slopes=P + 2)), BAD),
    (dict(score=osattn._Score(q_offset=(1 << 30) + 1)), BAD),
    (dict(score=rel_score(slopes=P)), BAD), (dict(score=rel_score(rel_map=None)), BAD),
    (dict(score=rel_score(rel_num=0)), BAD), (dict(score=rel_score(rel_range=0)), BAD),
    (dict(score=rel_score(rel_range=1025)), NOT), (dict(score=rel_score(softcap=5.0)), NOT),
    (dict(strides=((0, 64, 64), None, None, None)), BAD),
    (dict(strides=(None, None, (512, 68, 64), None)), BAD),
])
def test_fwd_mod_refusals(L, kw, expect):
    assert fwd(**kw) == expect


@pytest.mark.parametrize("kw,expect", [
    *[(dict(p=[P] * i + [None] + [P] * (8 - i)), BAD) for i in range(9)],
    (dict(p=[P] * 8 + [P + 4]), BAD), (dict(drel=P), BAD), (dict(score=rel_score()), BAD),
    (dict(ws=None), BAD), (dict(ws=P + 4), BAD), (dict(ws_bytes=4 * 8 * 4 - 1), BAD),
    (dict(score=rel_score(), drel=P, ws_bytes=(4 * 8 + 4 * 33) * 4 - 1), BAD),
    (dict(Hkv=3), BAD), (dict(d=80), NOT), (dict(dtype=osattn.FP32), NOT),
    (dict(strides=(None,) * 7 + ((512, 64, -64),)), BAD),
])
def test_bwd_mod_refusals(L, kw, expect):
    assert bwd(**kw) == expect


def test_sizes(L):
    assert osattn.bwd_mod_workspace_bytes(2, 3, 300, 500) == 2 * 3 * 300 * 4
    assert osattn.bwd_mod_workspace_bytes(2, 3, 300, 500, 16) == (2 * 3 * 300 + 2 * 3 * 4 * 33) * 4
    assert osattn.bwd_mod_workspace_bytes(2, 3, 0, 5) == 0
    assert L.osattn_mask_plan_bytes(2, 300) == 2 * (3 * 16 + 300 * 8)
    assert L.osattn_mask_plan_bytes(0, 300) == 0


@pytest.mark.parametrize("args", [
    (None, 1 << 20, 1, 8, 8, 0, 1, 0, None, None, None), (P + 4, 1 << 20, 1, 8, 8, 0, 1, 0, None, None, None),
    (P, 79, 1, 8, 8, 0, 1, 0, None, None, None), (P, 1 << 20, 0, 8, 8, 0, 1, 0, None, None, None),
    (P, 1 << 20, 1, 8, 0, 0, 1, 0, None, None, None), (P, 1 << 20, 1, 8, 8, 0, 1, -1, None, None, None),
    (P, 1 << 20, 1, 8, 8, 0, 0, 0, None, P, None), (P, 1 << 20, 1, 8, 8, 0, 1, 0, P + 2, None, None),
    (P, 1 << 20, 1, 8, 8, 0, 1, 0, None, None, P + 1), (P, 1 << 20, 1, 8, 8, -(1 << 30) - 1, 1, 0, None, None, None),
])
def test_mask_plan_refusals(L, args):
    assert L.osattn_mask_plan(*args, None) == BAD


def test_binding_refusals(L):
    q = torch.zeros(1, 4, 8, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        osattn.fwd_mod(q, q, q)  # not on a GPU
    with pytest.raises(TypeError):
        osattn.fwd_mod(q, q.float(), q)
    with pytest.raises(ValueError):
        osattn.fwd_mod(q, q[:, :3], q[:, :3])  # 3 key heads for 4 query heads
    with pytest.raises(ValueError):
        osattn.mask_plan(1, 8, 8, device="cpu")
    with pytest.raises(ValueError):
        osattn._view_strides(torch.zeros(1, 2, 64, 4).transpose(2, 3), "q")
    # the stride of an axis of length 1 says nothing
    s = osattn._view_strides(torch.zeros(8, 64, dtype=torch.bfloat16).as_strided((1, 1, 8, 64), (3, 0, 64, 1)), "q")
    assert list(s) == [512, 512, 64]
