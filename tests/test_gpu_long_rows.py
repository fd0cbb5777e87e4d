"""Rows of prompts of thousands of keys, sampled, against 64 bits key by key;
and tables, masks and page tables that are views of wider ones."""
import math

import pytest
import torch

import _rows
from attention_forward_online_gb300 import osattn

pytestmark = pytest.mark.gpu
DEV, F64 = "cuda", torch.float64
BF, FP = torch.bfloat16, torch.float16


def gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


@pytest.mark.parametrize("kind", ["plain", "cap", "slopes", "cap_slopes", "rel"])
@pytest.mark.parametrize("masks", [dict(causal=True), dict(causal=True, window=1500), {}, dict(causal=True, docs=900)],
                         ids=["causal", "window", "none", "documents"])
@pytest.mark.parametrize("dtype,d,N", [(BF, 128, 6500), (FP, 64, 9001)], ids=["bf16-128", "fp16-64"])
def test_sampled_rows(dtype, d, N, masks, kind):
    H, Hkv, g = 4, 2, gen(N)
    masks = dict(masks)
    q = (torch.randn(1, H, N, d, generator=g, device=DEV) * 2).to(dtype)
    k, v = (torch.randn(1, Hkv, N, d, generator=g, device=DEV).to(dtype) for _ in range(2))
    docs = masks.pop("docs", 0)
    ids = None
    if docs:
        ids = (torch.rand(1, N, generator=g, device=DEV) < 1 / docs).int().cumsum(1).int()
    plan = osattn.mask_plan(1, N, N, doc_ids=ids, device=DEV, **masks)
    cap = 30.0 if kind.startswith("cap") else 0.0
    slopes = torch.exp2(-2.0 * torch.arange(1, H + 1, device=DEV)) if kind.endswith("slopes") else None
    table = rel_map = None
    if kind == "rel":
        table, rel_map = torch.randn(32, H, generator=g, device=DEV).to(dtype), osattn.rel_buckets(32, 128).to(DEV)
    o, lse = osattn.fwd_mod(q, k, v, plan=plan, softcap=cap, slopes=slopes, rel_table=table, rel_map=rel_map)
    assert osattn.get_device_status() == osattn.OK
    at = torch.randperm(N, generator=g, device=DEV)[:60]
    at = torch.cat([at, torch.tensor([0, 1, 127, 128, 255, 256, N - 1], device=DEV)])
    gap = torch.arange(N, device=DEV)[None] - at[:, None]
    see = gap <= 0 if masks.get("causal") else torch.ones_like(gap, dtype=torch.bool)
    if "window" in masks:
        see &= gap.abs() < masks["window"]
    if docs:
        see &= ids[0][at][:, None] == ids[0][None]
    qq = q[0, :, at].to(F64)
    kk, vv = (x[0].to(F64).repeat_interleave(H // Hkv, 0) for x in (k, v))
    scale = 1 / math.sqrt(d)
    y = _rows.capped(scale * (qq @ kk.transpose(-1, -2)), cap)
    bias = torch.zeros(H, 1, 1, dtype=F64, device=DEV)
    if slopes is not None:
        bias = -slopes.to(F64)[:, None, None] * gap.abs()
    if table is not None:
        bias = table.to(F64)[rel_map.long()[gap.clamp(-128, 128) + 128]].permute(2, 0, 1)
    err = _rows.score_error(qq, kk, scale, y, bias) + 2.0 ** -20 * cap
    if slopes is not None:  # through the tensor core, see test_gpu_steep_slopes.py
        err = err + 3 * 2.0 ** -16 * slopes.to(F64)[:, None, None]
    _rows.check({"o": o[0, :, at], "lse": lse[0, :, at]}, _rows.rows(y + bias, see, err, vv, dtype))


def every_other(t):
    wide = torch.zeros(*t.shape[:-1], 2 * t.shape[-1], dtype=t.dtype, device=t.device)
    wide[..., ::2] = t
    return wide[..., ::2]


def test_views_of_tables_and_masks_say_the_same():
    B, H, N, g = 2, 4, 300, gen(1)
    q, do = (torch.randn(B, H, N, 64, generator=g, device=DEV).to(BF) for _ in range(2))
    k, v = (torch.randn(B, 2, N, 64, generator=g, device=DEV).to(BF) for _ in range(2))
    table = torch.randn(16, H, generator=g, device=DEV).to(BF)
    rel_map = osattn.rel_buckets(16, 60).to(DEV)
    docs = (torch.arange(N, device=DEV, dtype=torch.int32) // 70).repeat(B, 1)
    lens = torch.tensor([300, 211], dtype=torch.int32, device=DEV)
    slopes = torch.linspace(0.1, 0.9, H, device=DEV)

    def step(of, **mods):
        plan = osattn.mask_plan(B, N, N, causal=True, key_len=of(lens), prefix_len=of(lens // 3), doc_ids=of(docs))
        o, lse = osattn.fwd_mod(q, k, v, plan=plan, **mods)
        return (o, lse, *osattn.bwd_mod(q, k, v, o, lse, do, plan=plan, **mods))

    same = lambda t: t  # noqa: E731
    for a, b in zip(step(same, rel_table=table, rel_map=rel_map),
                    step(every_other, rel_table=table.t().contiguous().t(), rel_map=every_other(rel_map))):
        assert torch.equal(a, b)
    for a, b in zip(step(same, slopes=slopes), step(every_other, slopes=every_other(slopes))):
        assert torch.equal(a, b)
    per, T = 20, 4
    kp, vp = (torch.randn(B * per, 2, 16, 64, generator=g, device=DEV).to(BF) for _ in range(2))
    pages = torch.randperm(B * per, generator=g, device=DEV).int().reshape(B, per)
    wide = torch.full((B, 3 * per), -1, dtype=torch.int32, device=DEV)
    wide[:, :per] = pages
    mask = torch.tensor([[1, 3, 5, 9]] * B, device=DEV)
    for a, b in zip(osattn.tree_attn(q[:, :, :T], kp, vp, pages, lens, mask, slopes=slopes),
                    osattn.tree_attn(q[:, :, :T], kp, vp, wide[:, :per], every_other(lens), every_other(mask),
                                     slopes=every_other(slopes))):
        assert torch.equal(a, b)
    assert osattn.get_device_status() == osattn.OK
