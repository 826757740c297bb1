"""The measured cases of the attention operators: key ranges of a mask, per-head norms of queries and
keys with the position rotation, and masked attention with its gradients.

A case names its operator in "op":
  ranges       attention_key_ranges: documents, prefix, causal and window to one key interval per query
  rope         qk_norm_rope: RMSNorm of every query and key head and the rotation, one pass
  rope_grad    its backward: dq, dk and both gains' gradients
  attn         masked_attention_forward: O and the log-sum-exp of every row
  attn_step    forward and backward, as a training step calls them: O, lse, dq, dk, dv
Sizes follow the repository's attention workload (b2 s2048 h4096, 32 heads of 128) and sequence-parallel
block (b2 s4096 h4096), with grouped heads, narrower heads, ragged lengths and longer rows around them.
"""
import math
import random

import torch

own = False

BF16, F32 = "bf16", "f32"
_DTYPE = {BF16: torch.bfloat16, F32: torch.float32}
_EPS = 1e-5
_THETA = 10000.0


# ----------------------------------------------------------------------------- cases

def _ranges(name, b, s, docs, prefix, causal, window):
    return {"name": name, "op": "ranges", "b": b, "s": s, "docs": docs, "prefix": prefix, "causal": causal,
            "window": window}


def _rope(name, op, b, s, heads, kv, hd, rot, dtype, style, packed):
    return {"name": name, "op": op, "b": b, "s": s, "heads": heads, "kv": kv, "hd": hd, "rot": rot, "dtype": dtype,
            "style": style, "packed": packed}


def _attn(name, op, b, s, heads, kv, hd, docs=0, prefix=False, causal=True, window=0, cap=0.0, bias=False,
          packed=False):
    return {"name": name, "op": op, "b": b, "s": s, "heads": heads, "kv": kv, "hd": hd, "docs": docs, "prefix": prefix,
            "causal": causal, "window": window, "cap": cap, "bias": bias, "packed": packed}


def listed():
    return [
        # one batch of the attention workload, eight documents packed into each row
        _ranges("ranges-docs", 2, 2048, 8, False, True, 0),
        # a long packed row with a shared bidirectional prefix and a sliding window
        _ranges("ranges-long-prefix-window", 8, 8191, 40, True, True, 1024),
        # one new token for each of four sequences: launch latency
        _rope("rope-single-tokens", "rope", 4, 1, 32, 8, 128, 128, BF16, "half", False),
        # the attention workload's QKV matrix, heads packed as [q | k | v]
        _rope("rope-gpt", "rope", 2, 2048, 32, 32, 128, 128, BF16, "half", True),
        _rope("rope-grad-gpt", "rope_grad", 2, 2048, 32, 32, 128, 128, BF16, "half", True),
        # fp32, narrow heads, half of each head rotated in neighbouring pairs, odd length
        _rope("rope-grad-f32-ragged", "rope_grad", 3, 1111, 20, 4, 80, 40, F32, "interleaved", False),
        # a few short prompts with a prefix each, odd length, head width between the tile widths
        _attn("attn-short-prefix", "attn", 3, 77, 12, 4, 80, prefix=True),
        # the attention workload, causal, straight out of the packed QKV matrix
        _attn("attn-causal-gpt", "attn", 2, 2048, 32, 32, 128, packed=True),
        # a long row of packed documents with grouped heads and capped scores
        _attn("attn-docs-cap-long", "attn", 1, 8192, 32, 8, 128, docs=6, cap=30.0),
        # training step of the attention workload
        _attn("step-causal-gpt", "attn_step", 2, 2048, 32, 32, 128, packed=True),
        # distance bias and a sliding window on 64-wide heads, odd length
        _attn("step-bias-window", "attn_step", 2, 4001, 32, 32, 64, window=1024, bias=True),
        # the sequence-parallel block's length, documents, grouped heads and capped scores
        _attn("step-docs-cap-gqa", "attn_step", 2, 4096, 32, 8, 128, docs=3, cap=50.0),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _nameless(c):
    return {k: v for k, v in c.items() if k != "name"}


def draw(rng):
    op = rng.choice(["ranges", "rope", "rope_grad", "attn", "attn", "attn_step", "attn_step"])
    if op == "ranges":
        causal = rng.random() < 0.8
        return _nameless(_ranges("", rng.randint(1, 8), _log_int(rng, 200, 8191), rng.choice([2, 3, 17, 40]),
                                 causal and rng.random() < 0.5, causal, rng.choice([0, 0, 7, 100, 1024])))
    kv = rng.choice([1, 2, 3, 4, 8])
    heads = kv * rng.choice([1, 2, 4])
    hd = rng.choice([16, 40, 64, 64, 72, 80, 96, 128, 128, 128])
    packed = heads == kv and rng.random() < 0.7
    if op in ("rope", "rope_grad"):
        b = rng.choice([1, 2, 3, 5])
        s = _log_int(rng, 1, min(8192, 4096 * 4096 // (b * heads * hd)))
        return _nameless(_rope("", op, b, s, heads, kv, hd, rng.choice([hd, hd, hd // 4 * 2]),
                               rng.choice([BF16, BF16, F32]), rng.choice(["half", "interleaved"]), packed))
    b = rng.randint(1, 4)
    most = int(math.sqrt(2 * 32 * 4096 * 4096 / (b * heads)))
    # a step of one or two tokens has gradients that cancel to nothing, which no comparison can hold
    s = _log_int(rng, 1 if op == "attn" else 24, min(8192, most))
    causal = rng.random() < 0.75
    return _nameless(_attn("", op, b, s, heads, kv, hd, docs=rng.choice([0, 0, 2, 5]),
                           prefix=causal and rng.random() < 0.3, causal=causal,
                           window=rng.choice([0, 0, 0, 64, 1000]), cap=rng.choice([0.0, 0.0, 15.0, 50.0]),
                           bias=rng.random() < 0.3, packed=packed))


# ----------------------------------------------------------------------------- inputs

def _document_ids(c, seed=0):
    """Ids of the documents packed into each row, padding (id -1) behind the last one. Where attention runs over
    them the layout belongs to the case, so that its work is known."""
    rng = random.Random("%d %d %d %d" % (c["b"], c["s"], c["docs"], seed))
    rows = []
    for _ in range(c["b"]):
        end = c["s"] - rng.randint(0, c["s"] // 20)
        cuts = sorted(rng.randint(0, end) for _ in range(c["docs"] - 1))
        row = []
        for n, (lo, hi) in enumerate(zip([0] + cuts, cuts + [end])):
            row += [n] * (hi - lo)
        rows.append(row + [-1] * (c["s"] - end))
    return rows


def _prefix_lens(c, seed=0):
    rng = random.Random("%d %d prefix %d" % (c["b"], c["s"], seed))
    return [rng.randint(0, c["s"] // 2) for _ in range(c["b"])]


def _mask_inputs(c, seed=0):
    ids = prefix = None
    if c["docs"]:
        ids = torch.tensor(_document_ids(c, seed), dtype=torch.int32, device="cuda")
    if c["prefix"]:
        prefix = torch.tensor(_prefix_lens(c, seed), dtype=torch.int32, device="cuda")
    return ids, prefix


def _randn(gen, *shape):
    return torch.randn(*shape, generator=gen, device="cuda")


def _qkv(c, gen, dtype):
    """Queries, keys and values as a QKV GEMM leaves them: head by head [q | k | v] ("packed"), or all queries,
    then all keys, then all values."""
    b, s, heads, kv, hd = c["b"], c["s"], c["heads"], c["kv"], c["hd"]
    qkv = _randn(gen, b, s, (heads + 2 * kv) * hd).to(dtype)
    if c["packed"]:
        v5 = qkv.view(b, s, heads, 3, hd)
        return v5[:, :, :, 0], v5[:, :, :, 1], v5[:, :, :, 2]
    q, k, v = qkv.split([heads * hd, kv * hd, kv * hd], dim=-1)
    return q.unflatten(-1, (heads, hd)), k.unflatten(-1, (kv, hd)), v.unflatten(-1, (kv, hd))


def prepare(case, seed):
    c = case
    gen = torch.Generator("cuda").manual_seed(seed)
    if c["op"] == "ranges":
        ids, prefix = _mask_inputs(c, seed)
        return {"c": c, "ids": ids, "prefix": prefix}
    if c["op"] in ("rope", "rope_grad"):
        dtype = _DTYPE[c["dtype"]]
        q, k, _ = _qkv(c, gen, dtype)
        far = 4 * c["s"] + 64
        inv = _THETA ** (-torch.arange(0, c["rot"], 2, dtype=torch.float64, device="cuda") / c["rot"])
        ang = torch.arange(far, dtype=torch.float64, device="cuda")[:, None] * inv
        start = torch.randint(0, far - c["s"] + 1, (c["b"], 1), generator=gen, device="cuda")
        st = {"c": c, "q": q, "k": k, "gq": 1 + 0.1 * _randn(gen, c["hd"]), "gk": 1 + 0.1 * _randn(gen, c["hd"]),
              "cos": ang.cos().float(), "sin": ang.sin().float(),
              "pos": (start + torch.arange(c["s"], device="cuda")).int()}
        if c["op"] == "rope_grad":
            st["dq"] = _randn(gen, c["b"], c["s"], c["heads"], c["hd"]).to(dtype)
            st["dk"] = _randn(gen, c["b"], c["s"], c["kv"], c["hd"]).to(dtype)
        return st
    q, k, v = _qkv(c, gen, torch.bfloat16)
    ids, prefix = _mask_inputs(c)
    st = {"c": c, "q": q, "k": k, "v": v, "range": _plain_ranges(c, ids, prefix), "slopes": None}
    if c["bias"]:
        st["slopes"] = torch.exp2(-8.0 * torch.arange(1, c["heads"] + 1, device="cuda") / c["heads"])
    if c["op"] == "attn_step":
        st["do"] = _randn(gen, c["b"], c["s"], c["heads"], c["hd"]).to(torch.bfloat16)
    return st


# ----------------------------------------------------------------------------- plain forms

def _plain_ranges(c, ids, prefix):
    b, s, window = c["b"], c["s"], c["window"]
    i = torch.arange(s, device="cuda").expand(b, s)
    lo, hi = torch.zeros_like(i), torch.full_like(i, s)
    if ids is not None:
        new = torch.ones_like(ids, dtype=torch.bool)
        new[:, 1:] = ids[:, 1:] != ids[:, :-1]
        lo = torch.where(new, i, 0).cummax(dim=1).values
        last = torch.ones_like(new)
        last[:, :-1] = new[:, 1:]
        hi = torch.where(last, i + 1, s).flip(1).cummin(dim=1).values.flip(1)
    if c["causal"]:
        ahead = i + 1
        if prefix is not None:
            ahead = torch.maximum(ahead, prefix[:, None])
        hi = torch.minimum(hi, ahead)
    elif window:
        hi = torch.minimum(hi, i + window)
    if window:
        lo = torch.maximum(lo, i - window + 1)
    none = lo >= hi
    if ids is not None:
        none = none | (ids < 0)
    return torch.stack([torch.where(none, 0, lo), torch.where(none, 0, hi)], dim=-1).int()


def _rotate(x, cos, sin, style, back=False):
    rot = 2 * cos.shape[-1]
    if back:
        sin = -sin
    y = x.clone()
    if style == "half":
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        y[..., :rot // 2], y[..., rot // 2:rot] = a * cos - b * sin, b * cos + a * sin
    else:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        y[..., 0:rot:2], y[..., 1:rot:2] = a * cos - b * sin, b * cos + a * sin
    return y


def _plain_rope(x, gamma, cos, sin, style):
    xf = x.float()
    r = torch.rsqrt((xf * xf).mean(-1, keepdim=True) + _EPS)
    return _rotate(xf * r * gamma, cos, sin, style).to(x.dtype)


def _plain_rope_grad(x, gamma, cos, sin, style, dy):
    xf = x.float()
    r = torch.rsqrt((xf * xf).mean(-1, keepdim=True) + _EPS)
    xhat = xf * r
    du = _rotate(dy.float(), cos, sin, style, back=True)
    g = du * gamma
    dx = r * (g - xhat * (g * xhat).mean(-1, keepdim=True))
    return dx.to(x.dtype), (du * xhat).double().sum((0, 1, 2)).float()


def _plain_scores(st):
    """y = capped or plain scaled scores plus the distance bias [b, kv, r, s, s], -inf where hidden, and the
    derivative of the cap."""
    c = st["c"]
    b, s, heads, kv, hd = c["b"], c["s"], c["heads"], c["kv"], c["hd"]
    q = st["q"].float().view(b, s, kv, heads // kv, hd).permute(0, 2, 3, 1, 4)
    k = st["k"].float().permute(0, 2, 3, 1)[:, :, None]
    y = (q @ k) * hd ** -0.5
    slope = None
    if c["cap"]:
        t = torch.tanh(y / c["cap"])
        y, slope = c["cap"] * t, 1 - t * t
    j = torch.arange(s, device="cuda")
    if st["slopes"] is not None:
        y = y - st["slopes"].view(1, kv, -1, 1, 1) * (j[:, None] - j).abs()
    seen = (j >= st["range"][:, :, :1]) & (j < st["range"][:, :, 1:])
    return y.masked_fill(~seen[:, None, None], -math.inf), slope


def _heads_last(x, heads):
    """[b, kv, r, s, hd] -> [b, s, heads, hd]"""
    return x.permute(0, 3, 1, 2, 4).flatten(2, 3)


def _plain_attention(st):
    c = st["c"]
    y, slope = _plain_scores(st)
    top = y.amax(-1, keepdim=True)
    p = torch.exp(y - torch.where(top == -math.inf, 0, top))
    del y
    total = p.sum(-1, keepdim=True)
    lse = (top + total.log())[..., 0].flatten(1, 2)
    p = p / torch.where(total == 0, 1, total)
    v = st["v"].float().permute(0, 2, 1, 3)[:, :, None]
    o = p @ v
    out = (_heads_last(o, c["heads"]).to(torch.bfloat16), lse)
    if c["op"] == "attn":
        return out
    b, s, heads, kv, hd = c["b"], c["s"], c["heads"], c["kv"], c["hd"]
    do = st["do"].float().view(b, s, kv, heads // kv, hd).permute(0, 2, 3, 1, 4)
    dv = (p.transpose(-1, -2) @ do).sum(2)
    ds = p * (do @ v.transpose(-1, -2) - (do * o).sum(-1, keepdim=True))
    del p
    if slope is not None:
        ds = ds * slope
    ds = ds * hd ** -0.5
    q = st["q"].float().view(b, s, kv, heads // kv, hd).permute(0, 2, 3, 1, 4)
    k = st["k"].float().permute(0, 2, 1, 3)[:, :, None]
    dq = _heads_last(ds @ k, heads)
    dk = (ds.transpose(-1, -2) @ q).sum(2)
    return out + tuple(g.to(torch.bfloat16) for g in (dq, dk.transpose(1, 2), dv.transpose(1, 2)))


def _run_plain(st):
    c = st["c"]
    if c["op"] == "ranges":
        return _plain_ranges(c, st["ids"], st["prefix"])
    if c["op"] in ("rope", "rope_grad"):
        cos, sin = (st[n][st["pos"].long()][:, :, None] for n in ("cos", "sin"))
        if c["op"] == "rope":
            return tuple(_plain_rope(st[x], st["g" + x], cos, sin, c["style"]) for x in "qk")
        (dq, dgq), (dk, dgk) = (_plain_rope_grad(st[x], st["g" + x], cos, sin, c["style"], st["d" + x]) for x in "qk")
        return dq, dk, dgq, dgk
    return _plain_attention(st)


# ----------------------------------------------------------------------------- the framework's calls

def _run_own(st):
    import tensor_transformer_mlp_gb300 as tp

    c = st["c"]
    if c["op"] == "ranges":
        return tp.attention_key_ranges(c["b"], c["s"], doc_ids=st["ids"], prefix_len=st["prefix"], causal=c["causal"],
                                       window=c["window"], device="cuda")
    if c["op"] == "rope":
        return tp.qk_norm_rope(st["q"], st["k"], st["gq"], st["gk"], st["cos"], st["sin"], eps=_EPS,
                               positions=st["pos"], style=c["style"])
    if c["op"] == "rope_grad":
        return tp.qk_norm_rope_backward(st["q"], st["k"], st["gq"], st["gk"], st["cos"], st["sin"], st["dq"], st["dk"],
                                        eps=_EPS, positions=st["pos"], style=c["style"])
    o, lse = tp.masked_attention_forward(st["q"], st["k"], st["v"], st["range"], softcap=c["cap"], slopes=st["slopes"])
    if c["op"] == "attn":
        return o, lse
    return (o, lse) + tuple(tp.masked_attention_backward(st["q"], st["k"], st["v"], st["range"], o, lse, st["do"],
                                                         softcap=c["cap"], slopes=st["slopes"]))


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ----------------------------------------------------------------------------- work and exact values

def _intervals(c, all_ids, prefixes):
    """Each query's key interval [lo, hi) from the mask's definition, run of equal ids by run of equal ids."""
    rows = []
    for r in range(c["b"]):
        ids = all_ids[r] if all_ids is not None else [0] * c["s"]
        prefix, window = prefixes[r] if prefixes is not None else 0, c["window"]
        row, at = [], 0
        while at < c["s"]:
            end = at + 1
            while end < c["s"] and ids[end] == ids[at]:
                end += 1
            for i in range(at, end):
                lo = max(at, i - window + 1) if window else at
                hi = min(end, max(i + 1, prefix)) if c["causal"] else min(end, i + window) if window else end
                row.append((lo, hi) if lo < hi and ids[i] >= 0 else (0, 0))
            at = end
        rows.append(row)
    return rows


def work(case):
    c = case
    tokens = c["b"] * c["s"]
    if c["op"] == "ranges":
        return {"bytes": tokens * (8 + (4 if c["docs"] else 0)) + (4 * c["b"] if c["prefix"] else 0), "flops": 0}
    if c["op"] in ("rope", "rope_grad"):
        size = 2 if c["dtype"] == BF16 else 4
        values = tokens * (c["heads"] + c["kv"]) * c["hd"]
        tables = 4 * c["rot"] * min(tokens, 4 * c["s"] + 64) + 4 * tokens
        passes, flops = (2, 8) if c["op"] == "rope" else (3, 16)
        return {"bytes": values * size * passes + tables + 8 * c["hd"] * (passes - 1), "flops": values * flops}
    rows = _intervals(c, _document_ids(c) if c["docs"] else None, _prefix_lens(c) if c["prefix"] else None)
    pairs = sum(hi - lo for row in rows for lo, hi in row)
    q, kv = tokens * c["heads"] * c["hd"] * 2, tokens * c["kv"] * c["hd"] * 2
    nbytes = 2 * q + 2 * kv + 4 * tokens * c["heads"] + 8 * tokens  # q, k, v, o, lse and the key ranges
    products = 2  # q k^T and p v; the gradients need q k^T again, do v^T and three more
    if c["op"] == "attn_step":
        nbytes += 2 * q + 2 * kv
        products = 7
    return {"bytes": nbytes, "flops": 2.0 * products * c["hd"] * c["heads"] * pairs}


def _exact_attention(st):
    c = st["c"]
    b, s, heads, kv, hd = c["b"], c["s"], c["heads"], c["kv"], c["hd"]
    group = heads // kv
    dev = "cuda"
    j = torch.arange(s, device=dev)
    o = torch.zeros(b, s, heads, hd, dtype=torch.float64, device=dev)
    lse = torch.zeros(b, heads, s, dtype=torch.float64, device=dev)
    dq, dk, dv = torch.zeros_like(o), None, None
    step = c["op"] == "attn_step"
    if step:
        dk = torch.zeros(b, s, kv, hd, dtype=torch.float64, device=dev)
        dv = torch.zeros_like(dk)
    for bi in range(b):
        hidden = (j[None] < st["range"][bi, :, :1]) | (j[None] >= st["range"][bi, :, 1:])
        for h in range(heads):
            q, k, v = (st["q"][bi, :, h].double(), st["k"][bi, :, h // group].double(),
                       st["v"][bi, :, h // group].double())
            x = q @ k.T / math.sqrt(hd)
            t = None
            if c["cap"]:
                t = torch.tanh(x / c["cap"])
                x = t * c["cap"]
            if st["slopes"] is not None:
                x = x - st["slopes"][h].double() * (j[:, None] - j[None]).abs().double()
            x[hidden] = -math.inf
            row = torch.logsumexp(x, dim=-1)
            lse[bi, h] = row
            p = torch.exp(x - torch.where(row == -math.inf, 0, row)[:, None])
            o[bi, :, h] = p @ v
            if not step:
                continue
            do = st["do"][bi, :, h].double()
            dp = do @ v.T
            d = p * (dp - (p * dp).sum(-1, keepdim=True)) / math.sqrt(hd)
            if t is not None:
                d = d * (1 - t * t)
            dq[bi, :, h] = d @ k
            dk[bi, :, h // group] += d.T @ q
            dv[bi, :, h // group] += p.T @ do
    return (o, lse, dq, dk, dv) if step else (o, lse)


def _exact_rope(x, gamma, ang_cos, ang_sin, style, dy=None):
    """y, or the gradients from dy, of every head by explicit rotation matrices' entries in 64 bits."""
    x, gamma = x.double(), gamma.double()
    hd, rot = x.shape[-1], 2 * ang_cos.shape[-1]
    i = torch.arange(rot, device=x.device)
    if style == "half":
        partner, pair, sign = (i + rot // 2) % rot, i % (rot // 2), torch.where(i < rot // 2, -1.0, 1.0).double()
    else:
        partner, pair, sign = i ^ 1, i // 2, torch.where(i % 2 == 0, -1.0, 1.0).double()
    cos, sin = ang_cos.double()[..., pair], ang_sin.double()[..., pair] * sign
    scale = 1 / torch.sqrt(x.pow(2).sum(-1, keepdim=True) / hd + _EPS)
    if dy is None:
        u = x * scale * gamma
        return torch.cat([u[..., :rot] * cos + u[..., partner] * sin, u[..., rot:]], -1)
    dy = dy.double()
    du = torch.cat([dy[..., :rot] * cos - dy[..., partner] * sin, dy[..., rot:]], -1)
    g, xhat = du * gamma, x * scale
    dx = scale * (g - xhat * (g * xhat).sum(-1, keepdim=True) / hd)
    return dx, (du * xhat).sum((0, 1, 2))


def exact(case, seed):
    c = case
    st = prepare(c, seed)
    if c["op"] == "ranges":
        rows = _intervals(c, st["ids"].tolist() if st["ids"] is not None else None,
                          st["prefix"].tolist() if st["prefix"] is not None else None)
        return torch.tensor(rows, dtype=torch.int32)
    if c["op"] in ("rope", "rope_grad"):
        cos, sin = (st[n][st["pos"].long()][:, :, None] for n in ("cos", "sin"))
        if c["op"] == "rope":
            return tuple(_exact_rope(st[x], st["g" + x], cos, sin, c["style"]) for x in "qk")
        (dq, dgq), (dk, dgk) = (_exact_rope(st[x], st["g" + x], cos, sin, c["style"], st["d" + x]) for x in "qk")
        return dq, dk, dgq, dgk
    return _exact_attention(st)
