"""Plain 64-bit forms of modified-score attention for the tests, and how far a
16-bit kernel may be from them.

The bounds count roundings.  u is half a step of the element type
(finfo.eps / 2), and delta the error of a logit: the d-term product is summed
in fp32, an error below d 2^-24 sum |q_k k_k| scale, and the few fp32
operations on the score (cap, bias, base-2 conversion) err by at most 8 steps
of 2^-24 relative to the largest intermediate, taken as cap + |bias| + |y| and
(for |j - p| times a slope) slope |j - p|.  A probability is then off by at
most 2 delta relative (its logit and its row's sum), and the hardware's base-2
exponential by 2^-22.
  O:   P is rounded to the type as an operand, O at the end:
       |dO| <= (u + 2 delta + 2^-21) sum P |V| + u |O| (+ what P below fp16's
       smallest step 2^-24 loses: N 2^-25 max |V|, twice: P V and its row)
  dV:  the same with dO in place of V, over the rows of a group
  dY = P (dP - D): D is formed from the rounded O, so it errs by
       sum |dO| |error of O| =: eD;  |d dY| <= (2 delta + 2^-21) P (|dP| + |D|)
       + P (eD + d 2^-24 sum |dO| |V|)
  dS = dY (1 - t^2), t = tanh: 1 - t^2 errs by at most 2^-20 (absolute);
       rounded to the type as an operand: + u |dS| (+ 2^-25 for fp16)
  dQ, dK: sums of |d dS| |K| and |d dS| |Q|, plus u of the result
  dTable: the sum of |d dY| over a bucket's pairs, plus u of the result;
       every fp32 sum of n terms adds at most 2^-24 times (n terms deep at
       most, in blocks) the sum of magnitudes, taken as 2^-18 of it.
"""
import math

import torch

F64 = torch.float64
U = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
TINY = {torch.bfloat16: 0.0, torch.float16: 2.0 ** -25}


def visible(B, Nq, Nkv, causal=False, window=0, q_offset=0, key_len=None, prefix_len=None,
            doc_ids=None, device="cpu"):
    """bool [B, Nq, Nkv] from the definition of osattn_mask_plan."""
    p = torch.arange(Nq, device=device)[None, :, None] + q_offset
    j = torch.arange(Nkv, device=device)[None, None, :]
    see = torch.ones(B, Nq, Nkv, dtype=torch.bool, device=device)
    if key_len is not None:
        see &= j < torch.as_tensor(key_len, device=device)[:, None, None]
    if causal:
        past = j <= p
        if prefix_len is not None:
            past = past | (j < torch.as_tensor(prefix_len, device=device)[:, None, None])
        see &= past
    if window:
        see &= (j - p).abs() < window
    if doc_ids is not None:
        ids = torch.as_tensor(doc_ids, device=device)
        new = torch.ones_like(ids, dtype=torch.bool)
        new[:, 1:] = ids[:, 1:] != ids[:, :-1]
        run = new.long().cumsum(1)
        at = p[0, :, 0]
        ok = (at >= 0) & (at < Nkv)
        mine = torch.where(ok[None], run[:, at.clamp(0, Nkv - 1)], torch.full_like(run[:, :1], -1))
        mine = torch.where(ok[None] & (ids[:, at.clamp(0, Nkv - 1)] >= 0), mine, torch.full_like(mine, -1))
        see &= mine[:, :, None] == run[:, None, :]
    return see


def distance(Nq, Nkv, q_offset=0, device="cpu"):
    return (torch.arange(Nkv, device=device)[None, :]
            - torch.arange(Nq, device=device)[:, None] - q_offset)


def logits(q, k, scale, cap=0.0, slopes=None, table=None, rel_map=None, q_offset=0):
    """Modified scores [B, H, Nq, Nkv] in 64 bits; k with H heads."""
    y = scale * (q @ k.transpose(-1, -2))
    if cap:
        y = cap * torch.tanh(y / cap)
    gap = distance(q.shape[2], k.shape[2], q_offset, q.device)
    if slopes is not None:
        y = y - slopes[:, None, None] * gap.abs()
    if table is not None:
        R = rel_map.numel() // 2
        bucket = rel_map.long()[gap.clamp(-R, R) + R]
        live = (bucket >= 0) & (bucket < table.shape[0])
        bias = table[bucket.clamp(0, table.shape[0] - 1)].permute(2, 0, 1)
        y = y + torch.where(live, bias, torch.zeros_like(bias))
    return y


def softmax_out(y, see, v):
    """O, LSE, P; masked places hold nothing, rows that see nothing 0 and -inf."""
    y = torch.where(see, y, torch.full_like(y, -math.inf))
    top = y.amax(-1, keepdim=True)
    top = torch.where(torch.isfinite(top), top, torch.zeros_like(top)).detach()
    e = torch.exp(y - top)
    total = e.sum(-1, keepdim=True)
    p = e / torch.where(total > 0, total, torch.ones_like(total))
    lse = torch.where(total > 0, top + torch.log(torch.where(total > 0, total, torch.ones_like(total))),
                      torch.full_like(total, -math.inf)).squeeze(-1)
    return p @ v, lse, p


def reference(q, k, v, see, scale, do=None, cap=0.0, slopes=None, table=None, rel_map=None, q_offset=0):
    """Everything a call returns, in 64 bits, with the bounds above.  q, k, v,
    do, table are the 16-bit inputs.  -> dict name -> (value, bound)."""
    t = q.dtype
    u, tiny = U[t], TINY[t]
    H, Hkv = q.shape[1], k.shape[1]
    G = H // Hkv
    d, Nkv = q.shape[3], k.shape[2]
    leaf = [x.to(F64).requires_grad_(do is not None) for x in (q, k, v)]
    tab = None if table is None else table.to(F64).requires_grad_(do is not None)
    slo = None if slopes is None else slopes.to(F64)
    kk, vv = (x.repeat_interleave(G, 1) for x in leaf[1:])
    y = logits(leaf[0], kk, scale, cap, slo, tab, rel_map, q_offset)
    seen = see[:, None]
    o, lse, p = softmax_out(y, seen, vv)
    out = {}
    with torch.no_grad():
        s_abs = abs(scale) * (leaf[0].abs() @ kk.abs().transpose(-1, -2))
        gap = distance(q.shape[2], Nkv, q_offset, q.device).abs()
        big = y.abs() + cap + (0 if slo is None else slo[:, None, None] * gap) + s_abs
        delta = (d * 2.0 ** -24 * s_abs + 8 * 2.0 ** -24 * big)
        delta = torch.where(seen, delta, torch.zeros_like(delta)).amax(-1, keepdim=True)
        rel = 2 * delta + 2.0 ** -21
        lost = 2 * tiny * Nkv * (float(vv.abs().max()) + 1)
        eo = (u + rel) * (p @ vv.abs()) + lost + 2.0 ** -40
        out["o"] = (o.detach(), eo + u * o.abs() + tiny)
        fin = torch.isfinite(lse)
        out["lse"] = (lse.detach(), torch.where(fin, delta.squeeze(-1) + 2.0 ** -20
                                                + 2.0 ** -22 * lse.abs(), torch.zeros_like(lse)))
    if do is None:
        return out
    g64 = do.to(F64)
    wrt = leaf + ([] if tab is None else [tab])
    grads = torch.autograd.grad(o, wrt, g64)
    with torch.no_grad():
        dp = g64 @ vv.transpose(-1, -2)
        D = (g64 * o).sum(-1, keepdim=True)
        eD = (g64.abs() * (eo + u * o.abs() + tiny)).sum(-1, keepdim=True)
        edy = p * (rel * (dp.abs() + D.abs()) + eD + d * 2.0 ** -24 * (g64.abs() @ vv.abs().transpose(-1, -2)))
        dy = p * (dp - D)
        if cap:
            raw = scale * (leaf[0] @ kk.transpose(-1, -2))
            f = 1 - torch.tanh(raw / cap) ** 2
            eds = edy * f + dy.abs() * 2.0 ** -20
            ds = dy * f
        else:
            eds, ds = edy, dy
        eds = eds + u * ds.abs() + tiny
        few = 2.0 ** -18

        def shared(x):
            return x.reshape(x.shape[0], Hkv, G, *x.shape[2:]).sum(2)

        out["dq"] = (grads[0], abs(scale) * ((eds + few * ds.abs()) @ kk.abs()) + u * grads[0].abs() + tiny)
        out["dk"] = (grads[1], shared(abs(scale) * ((eds + few * ds.abs()).transpose(-1, -2) @ leaf[0].abs()))
                     + u * grads[1].abs() + tiny)
        ep = (u + rel + few) * p + tiny
        out["dv"] = (grads[2], shared(ep.transpose(-1, -2) @ g64.abs()) + u * grads[2].abs() + tiny)
        if tab is not None:
            R = rel_map.numel() // 2
            bucket = rel_map.long()[distance(q.shape[2], Nkv, q_offset, q.device).clamp(-R, R) + R]
            e = torch.zeros_like(grads[3])
            for n in range(tab.shape[0]):
                e[n] = ((edy + few * dy.abs()) * (bucket == n)).sum((0, 2, 3))
            out["drel"] = (grads[3], e + u * grads[3].abs() + tiny)
    return {n: (a.detach(), b.detach()) for n, (a, b) in out.items()}


def check(got, want, bound, name):
    got = got.detach().to(F64)
    assert got.shape == want.shape, name
    fin = torch.isfinite(want)
    assert torch.equal(got[~fin], want[~fin]), f"{name}: infinities differ"
    assert torch.isfinite(got[fin]).all(), f"{name}: not finite where the reference is"
    err, lim = (got - want)[fin].abs(), bound.expand_as(want)[fin]
    bad = err > lim
    assert not bad.any(), (f"{name}: {int(bad.sum())} of {err.numel()} over the bound, worst "
                           f"{float((err / lim.clamp(min=1e-30)).max()):.3g} times it")


def tree_reference(q, k_pages, v_pages, table, ctx, mask, scale, cap=0.0, slopes=None, window=0):
    """O, LSE of osattn_tree_attn with the bounds above: q [B, H, T, d], mask a
    list of T bit masks a sequence."""
    B, H, T, d = q.shape
    Hkv, page = k_pages.shape[1], k_pages.shape[2]
    u, tiny = U[q.dtype], TINY[q.dtype]
    o = torch.zeros(B, H, T, d, dtype=F64, device=q.device)
    lse = torch.full((B, H, T), -math.inf, dtype=F64, device=q.device)
    eo, el = torch.zeros_like(o), torch.zeros_like(lse)
    for b in range(B):
        n = ctx[b]
        pos = [n + max(bin(m).count("1") - 1, 0) for m in mask[b]]
        kpos = torch.tensor(list(range(n)) + pos)
        gap = (torch.tensor(pos)[:, None] - kpos[None]).abs()
        see = torch.zeros(T, n + T, dtype=torch.bool)
        for t, m in enumerate(mask[b]):
            see[t, :n] = m != 0
            for x in range(T):
                see[t, n + x] = bool((m >> x) & 1)
        if window:
            see &= gap < window
        gap, see = gap.to(q.device), see.to(q.device)
        keys = torch.arange(n + T, device=q.device)
        ids = table[b].long()[keys // page].clamp(0, k_pages.shape[0] - 1)
        used = see.any(0)
        k, v = (torch.where(used[:, None, None], x[ids, :, keys % page].to(F64), torch.zeros((), dtype=F64,
                                                                                             device=q.device))
                .transpose(0, 1).repeat_interleave(H // Hkv, 0) for x in (k_pages, v_pages))
        qq = q[b].to(F64)
        y = scale * (qq @ k.transpose(-1, -2))
        if cap:
            y = cap * torch.tanh(y / cap)
        fall = torch.zeros(H, 1, 1, dtype=F64, device=q.device) if slopes is None else slopes.to(F64)[:, None, None]
        y = y - fall * gap
        o[b], lse[b], p = softmax_out(y, see[None], v)
        s_abs = abs(scale) * (qq.abs() @ k.abs().transpose(-1, -2))
        big = y.abs() + cap + fall * gap + s_abs
        delta = torch.where(see[None], d * 2.0 ** -24 * s_abs + 8 * 2.0 ** -24 * big, torch.zeros_like(y))
        delta = delta.amax(-1, keepdim=True)
        rel = 2 * delta + 2.0 ** -21
        eo[b] = ((u + rel) * (p @ v.abs()) + 2 * tiny * (n + T) * (float(v.abs().max()) + 1) + 2.0 ** -40
                 + u * o[b].abs() + tiny)
        el[b] = delta.squeeze(-1) + 2.0 ** -20 + 2.0 ** -22 * lse[b].abs().nan_to_num(posinf=0)
    return {"o": (o, eo), "lse": (lse, el)}
