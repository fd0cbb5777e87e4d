"""Refusals and sizes of osattn_tree_attn, which need no GPU: every refused
call ends before a CUDA call."""
import ctypes
import math

import pytest
import torch

from attention_forward_online_gb300 import osattn

P = 0x10000
BAD, NOT = osattn.ERR_INVALID_ARG, osattn.ERR_UNSUPPORTED


@pytest.fixture(scope="module")
def L():
    from attention_forward_online_gb300 import _build

    _build.build()
    return osattn.lib()


def call(**kw):
    a = dict(p=[P] * 5, mask=P, o=P, lse=P, B=2, H=8, Hkv=2, T=5, d=64, pages=10, page=16, per=4,
             strides=(None,) * 4, scale=0.125, cap=0.0, slopes=None, window=0, dtype=osattn.BF16, ws=P,
             ws_bytes=1 << 30)
    a.update(kw)
    st = [None if s is None else (ctypes.c_int64 * 3)(*s) for s in a["strides"]]
    return osattn.lib().osattn_tree_attn(*a["p"], a["mask"], a["o"], a["lse"], a["B"], a["H"], a["Hkv"],
                                         a["T"], a["d"], a["pages"], a["page"], a["per"], *st, a["scale"],
                                         a["cap"], a["slopes"], a["window"], a["dtype"], a["ws"],
                                         a["ws_bytes"], None)


@pytest.mark.parametrize("kw,expect", [
    *[(dict(p=[P] * i + [None] + [P] * (4 - i)), BAD) for i in range(5)],
    (dict(o=None), BAD), (dict(lse=None), BAD), (dict(ws=None), BAD), (dict(ws=P + 8), BAD),
    (dict(mask=P + 4), BAD), (dict(slopes=P + 2), BAD), (dict(p=[P + 8] + [P] * 4), BAD),
    (dict(p=[P] * 3 + [P + 2, P]), BAD), (dict(o=P + 8), BAD),
    (dict(B=0), BAD), (dict(T=0), BAD), (dict(H=7), BAD), (dict(Hkv=0), BAD), (dict(pages=0), BAD),
    (dict(page=0), BAD), (dict(per=0), BAD), (dict(window=-1), BAD), (dict(scale=math.nan), BAD),
    (dict(cap=-2.0), BAD), (dict(cap=math.inf), BAD), (dict(cap=1e-4), BAD),
    (dict(T=65), NOT), (dict(H=258, Hkv=2), NOT), (dict(d=96), NOT), (dict(dtype=osattn.FP32), NOT),
    (dict(page=4), NOT), (dict(page=24), NOT), (dict(page=192), NOT),
    (dict(page=8, per=1, T=9), BAD),                     # the drafts do not fit the table
    (dict(page=128, per=(1 << 23) + 1), BAD),            # positions beyond 2^30
    (dict(page=128, per=1 << 20, B=1024, Hkv=8), BAD),   # list of tiles beyond 2^30
    (dict(strides=(None, (0, 64, 128), None, None)), BAD),
    (dict(strides=((640, 64, 132), None, None, None)), BAD),
])
def test_refusals(L, kw, expect):
    assert call(**kw) == expect


def test_workspaces_of_the_binding(L):
    for B, H, Hkv, T, d in [(1, 1, 1, 1, 64), (3, 8, 2, 5, 128), (4, 40, 8, 64, 64), (63, 128, 1, 2, 128),
                            (700, 96, 1, 3, 64)]:
        assert osattn._tree_workspace(B, H // Hkv, T, d) == osattn.tree_workspace_bytes(B, H, Hkv, T, d)
    for args in [(1, 1, 1, 1, 0), (2, 12, 381, 129, 0), (3, 4, 500, 128, 1024), (1, 16, 4096, 4097, 128)]:
        assert osattn._bwd_mod_workspace(*args) == osattn.bwd_mod_workspace_bytes(*args)


def test_workspace(L):
    rows = 2 * 160 * 5 * 4  # two partials a CTA, 5 tokens of 4 heads
    assert osattn.tree_workspace_bytes(2, 8, 2, 5, 64) == 16 + rows * 65 * 4
    assert osattn.tree_workspace_bytes(2, 8, 2, 64, 128) == 16 + 2 * 160 * 128 * 129 * 4
    assert osattn.tree_workspace_bytes(2, 8, 3, 5, 64) == 0
    assert osattn.tree_workspace_bytes(2, 8, 2, 65, 64) == 0
    assert call(ws_bytes=osattn.tree_workspace_bytes(2, 8, 2, 5, 64) - 1) == BAD


def test_binding_refusals(L):
    q = torch.zeros(1, 4, 1, 64, dtype=torch.bfloat16)
    k = torch.zeros(3, 2, 16, 64, dtype=torch.bfloat16)
    table, ctx = torch.zeros(1, 3, dtype=torch.int32), torch.zeros(1, dtype=torch.int32)
    with pytest.raises(ValueError):
        osattn.tree_attn(q, k, k, table, ctx)  # not on a GPU
    with pytest.raises(ValueError):
        osattn.tree_attn(q, k, k[:2], table, ctx)
    with pytest.raises(ValueError):
        osattn.tree_attn(q[:, :3], k, k, table, ctx)
    with pytest.raises(TypeError):
        osattn.tree_attn(q, k.float(), k.float(), table, ctx)
