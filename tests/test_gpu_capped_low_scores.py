"""fp16 rows all of whose scores lie far below 0: P has to keep fp16's precision
although no score is near the 0 that small capped scores are measured from."""
import math

import pytest
import torch

import _rows
from attention_forward_online_gb300 import osattn

pytestmark = pytest.mark.gpu
DEV, F64 = "cuda", torch.float64


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16], ids=["fp16", "bf16"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("near,far", [(-9.95, -17.6), (-7.5, -17.6), (-3.0, -9.9), (7.55, 7.7), (9.9, -9.9)])
def test_rows_of_low_scores(near, far, d, dtype):
    # one tile of keys at `near`, 32 tiles at `far`, whose weights of a thousandth
    # add up to some percent; V tells the two apart
    N, Nq, cap = 33 * 128, 130, 50.0
    g = torch.Generator(device=DEV).manual_seed(d)
    scale = 1 / math.sqrt(d)
    at = torch.full((N,), far, dtype=F64, device=DEV)
    at[:128] = near
    at += torch.rand(N, generator=g, device=DEV, dtype=F64) * 0.02
    q = torch.zeros(1, 1, Nq, d, dtype=dtype, device=DEV)
    k = torch.zeros(1, 1, N, d, dtype=dtype, device=DEV)
    q[..., 0] = 16.0
    k[0, 0, :, 0] = (at / (16.0 * scale)).to(dtype)
    v = torch.randn(1, 1, N, d, generator=g, device=DEV) * 0.1 - 1
    v[:, :, :128] += 2
    v = v.to(dtype)
    o, lse = osattn.fwd_mod(q, k, v, softcap=cap)
    assert osattn.get_device_status() == osattn.OK
    qq, kk, vv = (x.to(F64) for x in (q, k, v))
    y = _rows.capped(scale * (qq @ kk.transpose(-1, -2)), cap)
    err = _rows.score_error(qq, kk, scale, y, torch.zeros_like(y)) + 2.0 ** -20 * cap
    _rows.check({"o": o, "lse": lse}, _rows.rows(y, torch.ones_like(y, dtype=torch.bool), err, vv, dtype))
