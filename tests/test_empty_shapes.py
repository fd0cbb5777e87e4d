"""Shapes without heads or without elements, and a missing LSE, are refused as
values, like every other argument that does not fit."""
import pytest
import torch

from attention_forward_online_gb300 import osattn
from test_streams_host import Tensor, world  # noqa: F401

BF = torch.bfloat16


@pytest.mark.parametrize("H,Hkv,d", [(0, 2, 64), (2, 0, 64), (0, 0, 64), (2, 2, 0)])
def test_no_heads_or_elements(world, H, Hkv, d):  # noqa: F811
    q, kv = Tensor(world, (1, H, 4, d), BF, "q"), Tensor(world, (1, Hkv, 4, d), BF, "kv")
    lse = Tensor(world, (1, H, 4), torch.float32, "lse")
    with pytest.raises(ValueError):
        osattn.fwd_mod(q, kv, kv)
    with pytest.raises(ValueError):
        osattn.bwd_mod(q, kv, kv, q, lse, q)
    pages = Tensor(world, (3, Hkv, 16, d), BF, "pages")
    with pytest.raises(ValueError):
        osattn.tree_attn(q, pages, pages, Tensor(world, (1, 3), torch.int32, "table"),
                         Tensor(world, (1,), torch.int32, "ctx"))
    assert not [x for x in world.log if x[0].startswith("osattn_")]


def test_the_backward_pass_needs_the_lse(world):  # noqa: F811
    q = Tensor(world, (1, 2, 4, 64), BF, "q")
    with pytest.raises(ValueError):
        osattn.bwd_mod(q, q, q, q, None, q)
