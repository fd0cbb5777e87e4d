"""A plan may be dropped as soon as the calls that take it are queued, on
whichever stream they are."""
import pytest
import torch

from attention_forward_online_gb300 import osattn

pytestmark = pytest.mark.gpu
DEV, BF = "cuda", torch.bfloat16


@pytest.mark.parametrize("given", [True, False])
def test_a_plan_dropped_behind_a_call_on_another_stream(given):
    B, H, N = 1, 2, 700
    g = torch.Generator(device=DEV).manual_seed(1)
    q, k, v, do = (torch.randn(B, H, N, 64, generator=g, device=DEV).to(BF) for _ in range(4))

    def step(s):
        plan = osattn.mask_plan(B, N, N, causal=True, window=90, device=DEV)
        if s is not None:
            s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s if not given else None):
            if s is not None:
                with torch.cuda.stream(s):
                    torch.cuda._sleep(1 << 28)
            o, lse = osattn.fwd_mod(q, k, v, plan=plan, stream=s if given else None)
            grads = osattn.bwd_mod(q, k, v, o, lse, do, plan=plan, stream=s if given else None)
        size = plan.buffer.numel()
        del plan
        # plans of rows that see nothing, in whatever memory is free now
        taken = [torch.zeros(size, dtype=torch.uint8, device=DEV) for _ in range(64)]
        torch.cuda.synchronize()
        del taken
        return (o, lse, *grads)

    want = step(None)
    got = step(torch.cuda.Stream())
    assert osattn.get_device_status() == osattn.OK
    for a, b in zip(want, got):
        assert torch.equal(a, b)


def test_a_plan_made_before_the_capture_that_reads_it():
    B, H, N = 1, 2, 300
    g = torch.Generator(device=DEV).manual_seed(2)
    q, k, v, do = (torch.randn(B, H, N, 64, generator=g, device=DEV).to(BF) for _ in range(4))
    plan = osattn.mask_plan(B, N, N, causal=True, window=70, device=DEV)

    def step():
        o, lse = osattn.fwd_mod(q, k, v, plan=plan)
        return (o, lse, *osattn.bwd_mod(q, k, v, o, lse, do, plan=plan))

    want = step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for x in got:
        x.zero_()
    graph.replay()
    # made again in place: the next replay reads the new masks
    osattn.mask_plan(B, N, N, causal=True, window=20, device=DEV, out=plan)
    first = [x.clone() for x in got]
    graph.replay()
    again = step()
    torch.cuda.synchronize()
    for a, b, c, d in zip(want, first, again, got):
        assert torch.equal(a, b) and torch.equal(c, d)
    assert not torch.equal(want[0], again[0])
    del plan, graph, got
    torch.cuda.synchronize()
    assert osattn.get_device_status() == osattn.OK
