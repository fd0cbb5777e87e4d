"""Rotations in place with other strides, which need no GPU: threads would write rows that
others have not read yet, so the calls are refused."""
import pytest

from attention_forward_online_gb300 import osattn
from test_cache_api import BAD, L, P, append, rotary  # noqa: F401

CONTIGUOUS, SWAPPED = (8 * 5 * 64, 5 * 64, 64), (8 * 5 * 64, 64, 8 * 64)  # of B2 H8 N5 d64: by heads, by rows


@pytest.mark.parametrize("st", [(None, None, SWAPPED, None), (SWAPPED, None, None, None),
                                (SWAPPED, None, CONTIGUOUS, None), (CONTIGUOUS, None, (8 * 5 * 64 + 64, 5 * 64, 64), None),
                                ((0, 5 * 64, 64), None, CONTIGUOUS, None), (None, (2 * 5 * 64, 64, 2 * 64), None, None)])
def test_rotary(L, st):  # noqa: F811
    assert rotary(st=st) == BAD


@pytest.mark.parametrize("st", [(None, None, SWAPPED, None, None, None), (None,) * 5 + (SWAPPED,),
                                (None, None, CONTIGUOUS, None, None, SWAPPED)])
def test_append(L, st):  # noqa: F811
    assert append(st=st) == BAD
