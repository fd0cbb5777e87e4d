"""The gradients of a learned bias, and dK without a cap, are free of the error
that D = rowsum(dO O) takes from O's rounding to 16 bits.

V has a large common mean, so that O's rounding is large beside what tells the
keys apart.  The limits count roundings of independent values, each at most half
a step u of the type: the table's gradient is summed in fp32 and rounded once
(u of its norm); dK's dS are rounded before the product and the sum after it
(sqrt(2) u)."""
import pytest
import torch

import _mod_ref as R
from attention_forward_online_gb300 import osattn

F64 = torch.float64
H, N, D_HEAD = 4, 256, 64


def inputs(dtype, device, seed=7):
    g = torch.Generator().manual_seed(seed)
    q, k, v, do = (torch.randn(2, H, N, D_HEAD, generator=g) for _ in range(4))
    table = torch.randn(32, H, generator=g)
    return [x.to(dtype).to(device) for x in (q, k, v + 16, do, table)]


def exact(q, k, v, do, table, rel_map):
    see = torch.ones(2, N, N, dtype=torch.bool, device=q.device)
    want = R.reference(q, k, v, see, D_HEAD ** -0.5, do, 0.0, None, table, rel_map)
    return want["dk"][0], want["drel"][0]


def off(got, want):
    return float((got.to(F64) - want).norm() / want.norm())


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16], ids=["bf16", "fp16"])
def test_the_error_without_the_correction_is_beyond_the_limits(dtype):
    # the same computation in plain steps, with D as O's 16 bits give it and
    # with the row's sum of dY added to it
    q, k, v, do, table = inputs(dtype, "cpu")
    rel_map = osattn.rel_buckets(32, 100)
    dk, drel = exact(q, k, v, do, table, rel_map)
    qq, kk, vv, gg = (x.to(F64) for x in (q, k, v, do))
    y = R.logits(qq, kk, D_HEAD ** -0.5, table=table.to(F64), rel_map=rel_map)
    o, _, p = R.softmax_out(y, torch.ones_like(y, dtype=torch.bool), vv)
    dp = gg @ vv.transpose(-1, -2)
    D = (gg * o.to(dtype).to(F64)).sum(-1, keepdim=True)
    lost = (p * (dp - D)).sum(-1, keepdim=True)
    bucket = rel_map.long()[R.distance(N, N).clamp(-100, 100) + 100]
    hot = torch.nn.functional.one_hot(bucket.reshape(-1), 32).to(F64)

    def gradients(dy):
        dr = hot.t() @ dy.sum(0).reshape(H, -1).t()
        ds = dy.to(dtype).to(F64)
        return (D_HEAD ** -0.5 * ds.transpose(-1, -2) @ qq).to(dtype), dr.to(dtype)

    u = R.U[dtype]
    right, wrong = gradients(p * (dp - D - lost)), gradients(p * (dp - D))
    assert off(right[0], dk) < 1.5 * u and off(right[1], drel) < u
    assert off(wrong[0], dk) > 3 * u and off(wrong[1], drel) > 3 * u


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["rel", "plain"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16], ids=["bf16", "fp16"])
def test_gradients_have_the_correction(dtype, kind):
    q, k, v, do, table = inputs(dtype, "cuda")
    mods = {}
    if kind == "rel":
        mods = dict(rel_table=table, rel_map=osattn.rel_buckets(32, 100).cuda())
    o, lse = osattn.fwd_mod(q, k, v, **mods)
    grads = osattn.bwd_mod(q, k, v, o, lse, do, **mods)
    assert osattn.get_device_status() == osattn.OK
    u = R.U[dtype]
    if kind == "rel":
        dk, drel = exact(q, k, v, do, table, mods["rel_map"])
        assert off(grads[3], drel) < u
    else:
        see = torch.ones(2, N, N, dtype=torch.bool, device="cuda")
        dk = R.reference(q, k, v, see, D_HEAD ** -0.5, do)["dk"][0]
    assert off(grads[1], dk) < 1.5 * u
