"""Calls on a stream of their own while the current stream is still busy: the
copies of views that a call makes are in that stream's order."""
import math

import pytest
import torch

from attention_forward_online_gb300 import osattn

pytestmark = pytest.mark.gpu
DEV, BF = "cuda", torch.bfloat16


def on_a_stream(call):
    """call(stream) for the current stream at rest, then for another one while
    the current stream is busy; both results."""
    want = call(None)
    torch.cuda.synchronize()
    # memory that copies may land in holds something else before
    junk = [torch.full((n,), 0x7f, dtype=torch.uint8, device=DEV) for n in (64, 512, 4096, 1 << 16) for _ in range(8)]
    del junk
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    torch.cuda._sleep(1 << 28)  # about 0.15 s
    got = call(s)
    s.synchronize()
    torch.cuda.synchronize()
    assert osattn.get_device_status() == osattn.OK
    for a, b in zip(want, got):
        assert torch.equal(a, b)


def qkv(B, H, Hkv, N, d=64):
    g = torch.Generator(device=DEV).manual_seed(N)
    return [torch.randn(B, h, N, d, generator=g, device=DEV).to(BF) for h in (H, Hkv, Hkv, H)]


def every_other(t):
    wide = torch.zeros(*t.shape[:-1], 2 * t.shape[-1], dtype=t.dtype, device=t.device)
    wide[..., ::2] = t
    return wide[..., ::2]


def test_page_table_mask_lengths_and_slopes_as_views():
    B, H, T, page, per = 3, 8, 4, 16, 20
    g = torch.Generator(device=DEV).manual_seed(1)
    q = torch.randn(B, H, T, 64, generator=g, device=DEV).to(BF)
    kp, vp = (torch.randn(B * per, 2, page, 64, generator=g, device=DEV).to(BF) for _ in range(2))
    wide = torch.full((B, 3 * per), -1, dtype=torch.int32, device=DEV)
    wide[:, :per] = torch.arange(B * per, device=DEV).flip(0).reshape(B, per)
    ctx = every_other(torch.tensor([300, 17, 120], dtype=torch.int32, device=DEV))
    mask = every_other(torch.tensor([[1, 3, 5, 9]] * B, device=DEV))
    slopes = every_other(torch.linspace(0.1, 0.9, H, device=DEV))
    on_a_stream(lambda s: osattn.tree_attn(q, kp, vp, wide[:, :per], ctx, mask, slopes=slopes, window=90, stream=s))


def test_tables_and_masks_as_views():
    B, H, N = 2, 4, 300
    q, k, v, do = qkv(B, H, 2, N)
    table = torch.randn(H, 16, device=DEV).to(BF).t()
    rel_map = every_other(osattn.rel_buckets(16, 60).to(DEV))
    docs = every_other((torch.arange(N, device=DEV, dtype=torch.int32) // 70).repeat(B, 1))
    lens = every_other(torch.tensor([300, 211], dtype=torch.int32, device=DEV))

    def step(s):
        plan = osattn.mask_plan(B, N, N, key_len=lens, doc_ids=docs, stream=s)
        mods = dict(plan=plan, rel_table=table, rel_map=rel_map, stream=s)
        o, lse = osattn.fwd_mod(q, k, v, **mods)
        return (o, lse, *osattn.bwd_mod(q, k, v, o, lse, do, **mods))

    on_a_stream(step)


def test_key_lengths_of_the_plain_calls_as_views():
    B, H, N = 2, 4, 260
    q, k, v, do = qkv(B, H, H, N)
    lens = every_other(torch.tensor([260, 131], dtype=torch.int32, device=DEV))

    def step(s):
        o, lse = osattn.fwd(q, k, v, key_len=lens, stream=s)
        o2, lse2 = osattn.fwd_splitkv(q, k, v, 2, key_len=lens, stream=s)
        return (o, lse, o2, lse2, *osattn.bwd(q, k, v, o, lse, do, key_len=lens, stream=s))

    on_a_stream(step)


def test_host_memory_calls():
    B, H, N = 1, 4, 256
    q, k, v, do = (x.cpu().pin_memory() for x in qkv(B, H, H, N))
    x = torch.randn(64, 512).to(BF).pin_memory()

    def step(s):
        o, lse = osattn.fwd_offload(q, k, v, stream=s)
        y, rows = osattn.softmax_rows_offload(x, stream=s)
        (s or torch.cuda.current_stream()).synchronize()
        return (o, lse, y, rows, *osattn.bwd_offload(q, k, v, o, lse, do, stream=s))

    on_a_stream(step)


def test_a_call_on_a_stream_inside_a_graph():
    B, H, N = 1, 2, 200
    q, k, v, do = qkv(B, H, 1, N)
    lens = every_other(torch.tensor([150], dtype=torch.int32, device=DEV))
    side = torch.cuda.Stream()

    def step(s):
        plan = osattn.mask_plan(B, N, N, key_len=lens, stream=s)
        o, lse = osattn.fwd_mod(q, k, v, plan=plan, softcap=5.0, stream=s)
        return (o, lse, *osattn.bwd_mod(q, k, v, o, lse, do, plan=plan, softcap=5.0, stream=s))

    want = step(None)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        main = torch.cuda.current_stream()
        side.wait_stream(main)
        got = step(side)
        main.wait_stream(side)
    for x in got:
        x.fill_(math.nan)
    graph.replay()
    torch.cuda.synchronize()
    for a, b in zip(want, got):
        assert torch.equal(a, b)
