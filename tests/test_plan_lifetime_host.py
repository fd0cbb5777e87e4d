"""A plan's memory is the library's, so the library says where it is in use: on
every stream that a call reads it on, if that is not the one it was made on."""
import torch

from attention_forward_online_gb300 import osattn
from test_streams_host import MAIN, SIDE, Tensor, plan_of, qkv, stream, world  # noqa: F401


def marks(w):
    return [s for n, s in w.lent if n == "made"]


def test_a_plan_used_on_another_stream(world):  # noqa: F811
    q, k, v = qkv(world)
    lse = Tensor(world, (1, 4, 8), torch.float32, "lse")
    for use in (lambda plan, s: osattn.fwd_mod(q, k, v, plan=plan, out=q, lse=lse, stream=s),
                lambda plan, s: osattn.bwd_mod(q, k, v, q, lse, q, plan=plan, dq=q, dk=k, dv=v, workspace=q, stream=s)):
        plan = plan_of(world)
        world.lent.clear()
        use(plan, None)
        assert not marks(world)
        use(plan, stream(SIDE))
        assert SIDE in marks(world)
        # the same with the stream made the current one by the caller
        plan = plan_of(world)
        world.lent.clear()
        with torch.cuda.stream(stream(SIDE)):
            use(plan, None)
        assert SIDE in marks(world)


def test_a_plan_made_again_on_another_stream(world):  # noqa: F811
    plan = plan_of(world)
    world.lent.clear()
    osattn.mask_plan(1, 8, 8, device="cuda:0", out=plan, stream=stream(SIDE))
    assert SIDE in marks(world)
    # its memory still belongs to the stream that it was first made on
    q, k, v = qkv(world)
    world.lent.clear()
    osattn.fwd_mod(q, k, v, plan=plan, out=q, lse=Tensor(world, (1, 4, 8), torch.float32, "lse"), stream=stream(SIDE))
    assert SIDE in marks(world)
