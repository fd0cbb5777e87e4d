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
