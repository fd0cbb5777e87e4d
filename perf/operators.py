"""Timed cases of the attention operators whose scores are modified before
the softmax, of learned relative position biases, and of tree attention over
a paged cache: inputs, plain forms, the framework's calls, and 64-bit values.

`own` selects what run() does: False computes the operators in their plain
form with elementary torch operations in fp32, True makes the calls a user
makes.  A case is a dict of plain values; its `op` is one of

  mod    attention with a tanh cap, a distance slope, a sliding window,
         packed documents or a bidirectional prefix; forward, or a training
         step (forward and gradients)
  rel    attention with a learned bias by distance bucket; forward, or a
         training step that also returns the table's gradient
  tree   drafted tokens (one or a tree of them) of every sequence attending
         to its paged cache and to their own ancestors
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}

_MOD = dict(op="mod", B=1, H=8, Hkv=8, N=512, d=128, dtype="bf16", train=False, causal=True,
            cap=0.0, slopes=False, window=0, doc=0, prefix=0, ragged=False)
_REL = dict(op="rel", B=1, H=8, Hkv=8, N=512, d=64, dtype="bf16", train=False, causal=False,
            buckets=32, far=128, ragged=False)
_TREE = dict(op="tree", B=1, H=8, Hkv=8, T=1, d=128, dtype="bf16", ctx=512, page=64, cap=0.0,
             slopes=False, window=0)


def listed():
    return [
        # a prompt pass of a decoder with capped scores and shared key/value heads
        dict(_MOD, name="cap_prompt", H=32, N=8192, Hkv=8, cap=50.0),
        # a training step of a sliding-window layer of such a decoder
        dict(_MOD, name="cap_window_train", B=2, H=16, Hkv=4, N=4096, cap=50.0, window=1024,
             train=True),
        # a prompt batch of a decoder that has distance slopes in place of position embeddings
        dict(_MOD, name="slopes_prompt", B=4, H=16, Hkv=16, N=2048, d=64, dtype="fp16",
             slopes=True),
        # a training step on one long row packed with short documents
        dict(_MOD, name="documents_train", H=16, Hkv=16, N=8192, doc=700, train=True),
        # a small fine-tuning step: prefixes seen both ways, odd length, padded batch
        dict(_MOD, name="prefix_train_small", B=4, H=8, Hkv=2, N=381, d=64, dtype="fp16",
             prefix=100, ragged=True, train=True),
        # a training step of a text encoder with bucketed biases, padded batch
        dict(_REL, name="rel_encoder_train", B=8, H=12, Hkv=12, N=512, ragged=True, train=True),
        # a prompt pass of a decoder with one-sided buckets, odd length
        dict(_REL, name="rel_decoder_fwd", B=4, H=16, Hkv=16, N=1501, dtype="fp16", causal=True),
        # a long-document encoder's training step
        dict(_REL, name="rel_long_train", B=1, H=16, Hkv=16, N=4096, d=128, train=True),
        # one user's next token over a short context: latency
        dict(_TREE, name="decode_one", H=32, Hkv=8, ctx=700, page=16),
        # a serving batch's next tokens over ragged contexts
        dict(_TREE, name="decode_batch", B=64, H=32, Hkv=8, ctx=8192, page=64),
        # verification of drafted trees, capped scores
        dict(_TREE, name="tree_verify", B=8, H=32, Hkv=8, T=27, ctx=6000, page=32, cap=30.0),
        # wide trees over very long contexts with distance slopes
        dict(_TREE, name="tree_long", B=2, H=16, Hkv=2, T=64, d=64, dtype="fp16", ctx=100000,
             page=128, slopes=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["mod", "mod", "rel", "tree", "tree"])
    dtype, d = rng.choice(["bf16", "fp16"]), rng.choice([64, 128])
    if op == "tree":
        hkv, g = rng.choice([1, 2, 4, 8]), rng.choice([1, 2, 4, 5, 8])
        B, T = _log(rng, 1, 64), rng.choice([1, 1, _log(rng, 2, 64)])
        ctx = _log(rng, 30, 100000)
        while B * ctx * hkv * d > 64 * 8192 * 8 * 128 or B * ctx * hkv * g * T > 2 * 100000 * 16 * 64:
            B, ctx = max(1, B // 2), max(30, ctx * 2 // 3)
        return dict(_TREE, B=B, H=hkv * g, Hkv=hkv, T=T, d=d, dtype=dtype, ctx=ctx,
                    page=rng.choice([16, 32, 64, 128]), cap=rng.choice([0.0, 30.0]),
                    slopes=rng.random() < 0.3, window=rng.choice([0, 0, max(8, ctx // 3)]))
    hkv, g = rng.choice([1, 2, 4, 8]), rng.choice([1, 2, 4])
    B, N, train = _log(rng, 1, 8), _log(rng, 100, 8192), rng.random() < 0.6
    while B * hkv * g * N * N * (3 if train else 1) > 32 * 8192 * 8192:
        B, N = max(1, B // 2), N * 3 // 4
    base = dict(B=B, H=hkv * g, Hkv=hkv, N=N, d=d, dtype=dtype, train=train)
    if op == "rel":
        return dict(_REL, causal=rng.random() < 0.4, buckets=rng.choice([32, 64]),
                    far=rng.choice([64, 128, 200]), ragged=rng.random() < 0.5, **base)
    kind = rng.choice(["cap", "slopes", "window", "doc", "prefix"])
    return dict(_MOD, cap=rng.choice([0.0, 50.0]) if kind != "cap" else 30.0,
                slopes=kind == "slopes", window=max(16, N // 5) if kind == "window" else 0,
                doc=max(10, N // 9) if kind == "doc" else 0, prefix=N // 4 if kind == "prefix" else 0,
                causal=kind in ("window", "prefix") or rng.random() < 0.7,
                ragged=rng.random() < 0.3, **base)


# ------------------------------------------------------------------ inputs
def _bucket_map(buckets, far, both):
    """Bucket of each distance -far .. far (key position less query position):
    half of the buckets for exact small distances, the rest spaced by the
    logarithm up to `far`; with `both`, one half of all buckets per side."""
    rel = np.arange(-far, far + 1)
    n = buckets // 2 if both else buckets
    base = np.where(rel > 0, n, 0) if both else np.zeros_like(rel)
    dist = np.abs(rel) if both else np.maximum(-rel, 0)
    exact_n = n // 2
    big = exact_n + (np.log(np.maximum(dist, 1) / exact_n) / math.log(far / exact_n)
                     * (n - exact_n)).astype(np.int64)
    return torch.from_numpy((base + np.where(dist < exact_n, dist, np.minimum(big, n - 1))).astype(np.int32))


def prepare(case, seed):
    c = dict(case)
    g = torch.Generator(device=DEV).manual_seed(seed)
    h = np.random.RandomState(seed % (1 << 32))
    t = TYPES[c["dtype"]]
    B, H, Hkv, d = c["B"], c["H"], c["Hkv"], c["d"]

    def normal(*shape, std=1.0):
        return (torch.randn(*shape, generator=g, device=DEV) * std).to(t)

    def i32(a):
        return torch.as_tensor(np.asarray(a, dtype=np.int32)).to(DEV)

    s = {"case": c, "scale": 1.0 / math.sqrt(d)}
    # scores of standard deviation 2, as in trained heads that look at a few keys
    if c["op"] == "tree":
        T, page = c["T"], c["page"]
        lens = h.randint(c["ctx"] // 2, c["ctx"] + 1, B)
        lens[h.randint(B)] = c["ctx"]
        per = -(-(c["ctx"] + T) // page)
        pool = B * per
        s["q"] = normal(B, T, H, d, std=2.0).transpose(1, 2)
        s["k"] = normal(pool, page, Hkv, d).transpose(1, 2)
        s["v"] = normal(pool, page, Hkv, d).transpose(1, 2)
        s["table"] = i32(h.permutation(pool).reshape(B, per))
        s["ctx"] = i32(lens)
        # every draft's parent is the context or an earlier draft; a token sees its line
        masks = np.zeros((B, T), dtype=np.uint64)
        for b in range(B):
            for u in range(T):
                parent = h.randint(max(-1, u - 6), u) if u else -1
                masks[b, u] = (masks[b, parent] if parent >= 0 else np.uint64(0)) | np.uint64(1 << u)
        s["mask"] = torch.from_numpy(masks.view(np.int64)).to(DEV)
    else:
        N = c["N"]
        s["q"] = normal(B, N, H, d, std=2.0).transpose(1, 2)
        s["k"] = normal(B, N, Hkv, d).transpose(1, 2)
        s["v"] = normal(B, N, Hkv, d).transpose(1, 2)
        s["do"] = normal(B, N, H, d).transpose(1, 2) if c["train"] else None
        s["key_len"] = i32(h.randint(N // 2, N + 1, B)) if c["ragged"] else None
        s["doc"] = s["prefix"] = s["table"] = s["map"] = None
        if c["op"] == "rel":
            s["map"] = _bucket_map(c["buckets"], c["far"], not c["causal"]).to(DEV)
            s["table"] = normal(c["buckets"], H)
        else:
            if c["doc"]:
                s["doc"] = i32(np.cumsum(h.rand(B, N) < 1.0 / c["doc"], axis=1))
            if c["prefix"]:
                s["prefix"] = i32(h.randint(0, 2 * c["prefix"], B))
    s["slopes"] = None
    if c.get("slopes"):
        s["slopes"] = torch.exp2(-8.0 * torch.arange(1, H + 1, device=DEV, dtype=torch.float32) / H)
    return s


# ------------------------------------------------------------------ plain forms (fp32)
def _grouped(x, H):
    return x.float().repeat_interleave(H // x.shape[1], dim=1)


def _softmax_parts(logits, see):
    """P, LSE of logits where `see`; rows that see nothing give 0 and -inf."""
    logits = logits.masked_fill(~see, -math.inf)
    top = logits.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, torch.zeros_like(top), top)
    p = torch.exp(logits - top)
    total = p.sum(-1, keepdim=True)
    return p / torch.where(total > 0, total, torch.ones_like(total)), (top + torch.log(total)).squeeze(-1)


def _plain_dense(s):
    c = s["case"]
    H, N, t = c["H"], c["N"], s["q"].dtype
    q, k, v = s["q"].float(), _grouped(s["k"], H), _grouped(s["v"], H)
    i = torch.arange(N, device=DEV)[:, None]
    j = torch.arange(N, device=DEV)[None, :]
    see = torch.ones(1, N, N, dtype=torch.bool, device=DEV)
    if c["causal"]:
        past = (j <= i)[None]
        if s["prefix"] is not None:
            past = past | (j[None] < s["prefix"][:, None, None])
        see = see & past
    if c.get("window"):
        see = see & ((i - j).abs() < c["window"])[None]
    if s["doc"] is not None:
        see = see & (s["doc"][:, :, None] == s["doc"][:, None, :])
    if s["key_len"] is not None:
        see = see & (j[None] < s["key_len"][:, None, None])
    see = see[:, None]
    x = torch.matmul(q, k.transpose(-1, -2)) * s["scale"]
    slope = None
    cap = c.get("cap", 0.0)
    if cap:
        x = torch.tanh(x / cap)
        slope = 1 - x * x if c["train"] else None
        x = x * cap
    if s["slopes"] is not None:
        x = x - s["slopes"][:, None, None] * (i - j).abs()
    if c["op"] == "rel":
        far = c["far"]
        bucket = s["map"].long()[(j - i).clamp(-far, far) + far]
        x = x + s["table"].float()[bucket].permute(2, 0, 1)
    p, lse = _softmax_parts(x, see)
    del x
    o = torch.matmul(p, v)
    if not c["train"]:
        return o.to(t), lse
    do = s["do"].float()
    dv = torch.matmul(p.transpose(-1, -2), do)
    dx = p * (torch.matmul(do, v.transpose(-1, -2)) - (do * o).sum(-1, keepdim=True))
    del p
    out = [o.to(t)]
    drel = None
    if c["op"] == "rel":
        hot = (bucket.reshape(1, -1) == torch.arange(c["buckets"], device=DEV)[:, None]).float()
        drel = torch.matmul(hot, dx.sum(0).reshape(H, -1).t()).to(t)
        del hot
    if slope is not None:
        dx = dx * slope
    dx = dx * s["scale"]
    dq = torch.matmul(dx, k)
    dk = torch.matmul(dx.transpose(-1, -2), q)
    shared = (c["B"], c["Hkv"], H // c["Hkv"], N, c["d"])
    out += [dq.to(t), dk.reshape(shared).sum(2).to(t), dv.reshape(shared).sum(2).to(t)]
    return tuple(out) if drel is None else tuple(out) + (drel,)


def _plain_tree(s):
    c = s["case"]
    B, H, T, d = c["B"], c["H"], c["T"], c["d"]
    t = s["q"].dtype
    per, page = s["table"].shape[1], c["page"]
    L = per * page

    def gathered(x):  # [pages, Hkv, page, d] -> [B, Hkv, L, d]
        return x[s["table"].long()].transpose(1, 2).reshape(B, c["Hkv"], L, d).float()

    q = s["q"].float().reshape(B, c["Hkv"], H // c["Hkv"] * T, d)
    k, v = gathered(s["k"]), gathered(s["v"])
    ctx = s["ctx"].long()[:, None, None]
    j = torch.arange(L, device=DEV)[None, None, :]
    u = j - ctx  # the draft that a key behind the context is
    inside = (u >= 0) & (u < T)
    line = (s["mask"][:, :, None] >> u.clamp(0, T - 1)) & 1
    see = (u < 0) | (inside & (line == 1))  # [B, T, L]
    bits = torch.arange(T, device=DEV)
    depth = ((s["mask"][:, :, None] >> bits) & 1).sum(-1) - 1  # [B, T]
    qpos = ctx + depth[:, :, None]
    kpos = torch.where(inside, ctx + torch.gather(depth, 1, u.clamp(0, T - 1).reshape(B, L))[:, None], j)
    dist = (qpos - kpos).abs()  # [B, T, L]
    if c["window"]:
        see = see & (dist < c["window"])
    x = (torch.matmul(q, k.transpose(-1, -2)) * s["scale"]).reshape(B, H, T, L)
    if c["cap"]:
        x = torch.tanh(x / c["cap"]) * c["cap"]
    if s["slopes"] is not None:
        x = x - s["slopes"][:, None, None] * dist[:, None]
    p, lse = _softmax_parts(x, see[:, None])
    o = torch.matmul(p.reshape(B, c["Hkv"], -1, L), v).reshape(B, H, T, d)
    return o.to(t), lse


# ------------------------------------------------------------------ the framework's calls
def _own(s):
    from attention_forward_online_gb300 import osattn

    c = s["case"]
    if c["op"] == "tree":
        return osattn.tree_attn(s["q"], s["k"], s["v"], s["table"], s["ctx"], s["mask"],
                                scale=s["scale"], softcap=c["cap"], slopes=s["slopes"],
                                window=c["window"])
    plan = osattn.mask_plan(c["B"], c["N"], c["N"], causal=c["causal"], window=c.get("window", 0),
                            key_len=s["key_len"], prefix_len=s["prefix"], doc_ids=s["doc"])
    mods = dict(scale=s["scale"], plan=plan, softcap=c.get("cap", 0.0), slopes=s["slopes"],
                rel_table=s["table"], rel_map=s["map"])
    o, lse = osattn.fwd_mod(s["q"], s["k"], s["v"], **mods)
    if not c["train"]:
        return o, lse
    return (o, *osattn.bwd_mod(s["q"], s["k"], s["v"], o, lse, s["do"], **mods))


def run(state):
    if own:
        return _own(state)
    return _plain_tree(state) if state["case"]["op"] == "tree" else _plain_dense(state)


# ------------------------------------------------------------------ floors
def _pairs(c):
    """Expected query-key pairs of one head of one batch entry."""
    N = c["N"]
    n = N * (N + 1) / 2 if c["causal"] else N * N
    if c.get("window"):
        w = min(c["window"], N)
        n = min(n, N * w * (1 if c["causal"] else 2))
    if c.get("doc"):
        n = min(n, N * c["doc"] * (1 if c["causal"] else 2))
    if c.get("prefix"):
        n = n + c["prefix"] * c["prefix"] / 2
    if c["ragged"]:
        n = n * (0.75 if not c["causal"] else 0.9)
    return n


def work(case):
    c = case
    H, Hkv, d = c["H"], c["Hkv"], c["d"]
    if c["op"] == "tree":
        keys = c["B"] * (0.75 * c["ctx"] + c["T"])
        if c["window"]:
            keys = min(keys, c["B"] * (c["window"] + c["T"]))
        return {"bytes": 2 * (2 * keys * Hkv * d + 2 * c["B"] * c["T"] * H * d) + 4 * c["B"] * H * c["T"],
                "flops": 4.0 * keys * c["T"] * H * d}
    rows_q, rows_k = c["B"] * H * c["N"], c["B"] * Hkv * c["N"]
    flops = 4.0 * d * c["B"] * H * _pairs(c)
    data = 2 * d * (2 * rows_q + 2 * rows_k) + 4 * rows_q
    if c["train"]:  # dO read and dQ, dK, dV written besides; five more products of S's size
        flops *= 3.5
        data += 2 * d * (2 * rows_q + 2 * rows_k)
    return {"bytes": data, "flops": flops}


# ------------------------------------------------------------------ 64-bit values
def _exact_head(q, k, v, bias, see, scale, cap):
    """O, LSE of one head in 64 bits; differentiable."""
    x = scale * (q @ k.T)
    if cap:
        x = cap * torch.tanh(x / cap)
    x = x if bias is None else x + bias
    empty = ~see.any(1)
    x = torch.where(see, x, torch.full((), -1e300, dtype=torch.float64, device=DEV))
    lse = torch.logsumexp(x, 1)
    w = torch.where(see, torch.softmax(x, 1), torch.zeros((), dtype=torch.float64, device=DEV))
    return w @ v, torch.where(empty, torch.full_like(lse, -math.inf), lse)


def exact(case, seed):
    s = prepare(case, seed)
    c = s["case"]
    B, H, Hkv = c["B"], c["H"], c["Hkv"]
    per = H // Hkv
    f64 = dict(dtype=torch.float64, device=DEV)
    if c["op"] == "tree":
        T, page = c["T"], c["page"]
        o = torch.zeros(B, H, T, c["d"], **f64)
        lse = torch.zeros(B, H, T, **f64)
        masks = s["mask"].cpu().numpy().view(np.uint64)
        for b in range(B):
            n = int(s["ctx"][b])
            pages = s["table"][b].long()
            seen = np.array([[(int(m) >> u) & 1 for u in range(T)] for m in masks[b]], dtype=bool)
            pos = n + seen.sum(1) - 1
            kpos = torch.from_numpy(np.concatenate([np.arange(n), pos])).to(DEV)
            gap = (torch.from_numpy(pos).to(DEV)[:, None] - kpos[None, :]).abs()
            see = torch.ones(T, n + T, dtype=torch.bool, device=DEV)
            see[:, n:] = torch.from_numpy(seen).to(DEV)
            if c["window"]:
                see &= gap < c["window"]
            for h in range(H):
                k = s["k"][pages, h // per].reshape(-1, c["d"])[: n + T].double()
                v = s["v"][pages, h // per].reshape(-1, c["d"])[: n + T].double()
                bias = None if s["slopes"] is None else -s["slopes"][h].double() * gap
                o[b, h], lse[b, h] = _exact_head(s["q"][b, h].double(), k, v, bias, see, s["scale"], c["cap"])
        return o, lse
    N = c["N"]
    at = torch.arange(N, device=DEV)
    gap = at[None, :] - at[:, None]
    o = torch.zeros(B, H, N, c["d"], **f64)
    lse = torch.zeros(B, H, N, **f64)
    dq, dk, dv = torch.zeros_like(o), torch.zeros(B, Hkv, N, c["d"], **f64), torch.zeros(B, Hkv, N, c["d"], **f64)
    drel = None
    if c["op"] == "rel":
        drel = torch.zeros(c["buckets"], H, **f64)
        where = s["map"].long()[gap.clamp(-c["far"], c["far"]) + c["far"]]
    for b in range(B):
        see = torch.ones(N, N, dtype=torch.bool, device=DEV)
        if c["causal"]:
            see = gap <= 0
            if s["prefix"] is not None:
                see = see | (at < s["prefix"][b])[None, :]
        if c.get("window"):
            see = see & (gap.abs() < c["window"])
        if s["doc"] is not None:
            see = see & (s["doc"][b][None, :] == s["doc"][b][:, None])
        if s["key_len"] is not None:
            see = see & (at < s["key_len"][b])[None, :]
        for h in range(H):
            q, k, v = (x.double().requires_grad_(c["train"]) for x in
                       (s["q"][b, h], s["k"][b, h // per], s["v"][b, h // per]))
            bias = row = None
            if s["slopes"] is not None:
                bias = -s["slopes"][h].double() * gap.abs()
            if drel is not None:
                row = s["table"][:, h].double()
                bias = row[where].requires_grad_(c["train"])
            oh, lh = _exact_head(q, k, v, bias, see, s["scale"], c.get("cap", 0.0))
            o[b, h], lse[b, h] = oh.detach(), lh.detach()
            if c["train"]:
                wrt = [q, k, v] + ([bias] if drel is not None else [])
                got = torch.autograd.grad(oh, wrt, s["do"][b, h].double())
                dq[b, h] = got[0]
                dk[b, h // per] += got[1]
                dv[b, h // per] += got[2]
                if drel is not None:
                    drel[:, h] += torch.bincount(where.reshape(-1), got[3].reshape(-1), c["buckets"])
    if not c["train"]:
        return o, lse
    return (o, dq, dk, dv) if drel is None else (o, dq, dk, dv, drel)
