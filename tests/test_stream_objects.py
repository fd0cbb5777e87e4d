"""A call takes any object with a stream's handle, and refuses a stream of
another device."""
import types

import pytest
import torch

from attention_forward_online_gb300 import osattn
from test_streams_host import SIDE, Tensor, stream, world  # noqa: F401

BF = torch.bfloat16


def calls(w, s):
    q = Tensor(w, (1, 2, 8, 64), BF, "q")
    return [lambda: osattn.fwd(q, q, q, stream=s), lambda: osattn.fwd_mod(q, q, q, stream=s),
            lambda: osattn.softmax_rows(Tensor(w, (4, 8), BF, "x"), stream=s)]


def test_a_handle_is_enough(world, monkeypatch):  # noqa: F811
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda handle, device: stream(handle))
    for call in calls(world, types.SimpleNamespace(cuda_stream=SIDE)):
        world.log.clear()
        call()
        assert len(world.log) > 1 and {s for _, s in world.log} == {SIDE}


def test_a_stream_of_another_device(world):  # noqa: F811
    other = types.SimpleNamespace(cuda_stream=SIDE, device_index=1)
    for call in calls(world, other):
        with pytest.raises(ValueError):
            call()
    assert not world.log
