"""64-bit rows of softmax attention with bounds that go key by key: where
_mod_ref.py takes the worst logit error of a row for all of its keys, here each
key's error counts with its own weight, so that a key next to the query is not
excused by one far away.

err_j bounds the error of logit j.  With weights P:
  LSE: sum P err (first order; err is below 0.05 wherever this is used, so the
       second order is within a tenth of it), plus 2^-20 for the base-2
       exponentials (2^-22 each), the fp32 sums and the logarithm's argument,
       plus 2^-22 |LSE| for its conversions
  O:   sum P (err_j + sum P err) |V_j| by the weights, (u + 2^-21) sum P |V| by
       the rounding of P to the type, what P below fp16's smallest step loses
       (half a step 2^-25 a key, once in the products and once in the sum,
       against a row sum of 1/2 or more), and half a step of the result
"""
import torch

import _mod_ref as R

F64 = torch.float64


def score_error(q, k, scale, y, bias):
    """Error of the logits y from q, k (64-bit copies of the 16-bit inputs): the
    product is summed in fp32, d 2^-24 of the sum of magnitudes, and the
    operations on the score are off by at most 8 steps of 2^-24 of the largest
    intermediate; no cap's size enters."""
    s_abs = abs(scale) * (q.abs() @ k.abs().transpose(-1, -2))
    return q.shape[-1] * 2.0 ** -24 * s_abs + 8 * 2.0 ** -24 * (y.abs() + bias.abs() + s_abs)


def rows(y, see, err, v, dtype):
    """{"o": (value, bound), "lse": ...}: y, err [..., Nq, Nk], see likewise, v [..., Nk, d]."""
    u, tiny = R.U[dtype], R.TINY[dtype]
    o, lse, p = R.softmax_out(y, see, v)
    err = torch.where(see, err, torch.zeros_like(err))
    mean = (p * err).sum(-1, keepdim=True)
    most = float(v.abs().max())
    eo = 1.1 * ((p * (err + mean)) @ v.abs()) + (u + 2.0 ** -21) * (p @ v.abs())
    eo = eo + 4 * tiny * y.shape[-1] * (most + 1) + u * o.abs() + tiny + 2.0 ** -40
    fin = torch.isfinite(lse)
    el = 1.1 * mean.squeeze(-1) + 2.0 ** -20 + 2.0 ** -22 * torch.where(fin, lse, torch.zeros_like(lse)).abs()
    return {"o": (o, eo), "lse": (lse, el)}


def check(got, want):
    for n, (value, bound) in want.items():
        R.check(got[n], value, bound, n)


def capped(x, cap):
    return cap * torch.tanh(x / cap) if cap else x

