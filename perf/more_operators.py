"""The measured cases of the gated feed-forward block and of the norms around a block.

A case names its operator in "op":
  gated               gated_forward: Z = X A, Y = act(Z_gate) * Z_up, O = Y B (with "save" also Z and Y for the backward)
  gated_grad          gated_backward from the saved Z and Y: dX, dA and dB, the weights' gradients in the operands' type
  residual_norm       residual_norm: r = alpha x + gate * rmsnorm(y), u = rmsnorm(r), one pass
  residual_norm_grad  its backward: dx, dy, both gains' gradients and the gate's
Sizes follow the repository's workloads (single block n512 d1024 m4096 t2, GPT MLP n8192 d4096 m16384 t8, sequence-parallel
block b2 s4096 h4096) with single tokens, small batches of them, ragged sizes and narrower rows around them.
"""
import math
import random

import torch

own = False

BF16, F32 = "bf16", "f32"
_DTYPE = {BF16: torch.bfloat16, F32: torch.float32}
_EPS = 1e-5


# ----------------------------------------------------------------------------- cases

def _gated(name, op, n, d, m, t, act, save=False):
    return {"name": name, "op": op, "n": n, "d": d, "m": m, "t": t, "act": act, "save": save}


def _norm(name, op, b, s, h, dtype, post=True, pre=True, gate="none", alpha=1.0):
    return {"name": name, "op": op, "b": b, "s": s, "h": h, "dtype": dtype, "post": post, "pre": pre, "gate": gate,
            "alpha": alpha}


def listed():
    return [
        # one new token for each of four sequences through a layer of the GPT MLP's size: the weights' bytes
        _gated("gated-single-tokens", "gated", 4, 4096, 16384, 8, "silu"),
        # a short prompt through the single block: launch latency
        _gated("gated-short-prompt", "gated", 37, 1024, 4096, 2, "gelu_tanh"),
        # a step of serving with some two hundred sequences at once
        _gated("gated-serving-batch", "gated", 200, 4096, 16384, 8, "silu"),
        # training forward of the GPT MLP's tokens, Z and Y kept
        _gated("gated-gpt", "gated", 8192, 4096, 16384, 8, "silu", save=True),
        # backward of the single block
        _gated("gated-grad-single-block", "gated_grad", 512, 1024, 4096, 2, "gelu_tanh"),
        # odd sizes: ragged tiles in every dimension, shards that end inside a tile
        _gated("gated-grad-ragged", "gated_grad", 1111, 1000, 2736, 2, "gelu_erf"),
        # backward of the GPT MLP
        _gated("gated-grad-gpt", "gated_grad", 8192, 4096, 16384, 8, "silu"),
        # four single tokens, a gate for each sequence: launch latency
        _norm("norm-single-tokens", "residual_norm", 4, 1, 4096, BF16, gate="sequence"),
        # the sequence-parallel block's activations, a learned gate and a residual scale
        _norm("norm-sp-block", "residual_norm", 2, 4096, 4096, BF16, gate="vector", alpha=1.5),
        # fp32, odd length and width
        _norm("norm-f32-ragged", "residual_norm", 3, 1111, 1608, F32, gate="sequence", alpha=0.5),
        # backward at the sequence-parallel block's size, a gate for each sequence
        _norm("norm-grad-sp-block", "residual_norm_grad", 2, 4096, 4096, BF16, gate="sequence"),
        # its fp32 form, ragged, a learned gate and a residual scale
        _norm("norm-grad-f32-ragged", "residual_norm_grad", 3, 1111, 1608, F32, gate="vector", alpha=0.5),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["gated", "gated", "gated_grad", "gated_grad", "residual_norm", "residual_norm_grad"])
    if op.startswith("gated"):
        n = _log_int(rng, 1, 8192)
        d = 8 * _log_int(rng, 16, 512)
        t = rng.choice([1, 1, 2, 4, 8])
        m = 8 * t * max(1, round(d * rng.uniform(1.0, 4.0) / (8 * t)))
        c = _gated("", op, n, d, m, t, rng.choice(["silu", "silu", "gelu_tanh", "gelu_erf"]),
                   save=op == "gated" and rng.random() < 0.5)
    else:
        h = 8 * _log_int(rng, 8, 1024)
        b = rng.choice([1, 2, 3, 7, 40])
        s = _log_int(rng, 1, max(1, min(8192, 8192 * 4096 // (b * h))))
        dtype = rng.choice([BF16, BF16, F32])
        c = _norm("", op, b, s, h, dtype, post=rng.random() < 0.8, pre=rng.random() < 0.8,
                  gate=rng.choice(["none", "vector", "sequence"]), alpha=rng.choice([1.0, 1.0, 0.7, 2.0]))
    del c["name"]
    return c


# ----------------------------------------------------------------------------- inputs

def _randn(gen, *shape):
    return torch.randn(*shape, generator=gen, device="cuda")


def _shards(c, z):
    """The gate and up columns [..., m] of a [..., 2 m] matrix whose shards hold [gate | up] each."""
    v = z.unflatten(-1, (c["t"], 2, c["m"] // c["t"]))
    return v[..., 0, :].flatten(-2), v[..., 1, :].flatten(-2)


def _join(c, gate, up):
    """The inverse of _shards."""
    parts = [x.unflatten(-1, (c["t"], c["m"] // c["t"])) for x in (gate, up)]
    return torch.stack(parts, dim=-2).flatten(-3)


def prepare(case, seed):
    c = case
    gen = torch.Generator("cuda").manual_seed(seed)
    if c["op"].startswith("gated"):
        n, d, m = c["n"], c["d"], c["m"]
        st = {"c": c, "X": _randn(gen, n, d).to(torch.bfloat16),
              "A": (d ** -0.5 * _randn(gen, d, 2 * m)).to(torch.bfloat16),
              "B": (m ** -0.5 * _randn(gen, m, d)).to(torch.bfloat16)}
        if c["op"] == "gated_grad":  # what the forward kept
            st["G"] = _randn(gen, n, d).to(torch.bfloat16)
            st["Z"] = st["X"] @ st["A"]
            gate, up = _shards(c, st["Z"].float())
            st["Y"] = (_act(c, gate) * up).to(torch.bfloat16)
        return st
    dtype, shape, h = _DTYPE[c["dtype"]], (c["b"], c["s"], c["h"]), c["h"]
    x, y = _randn(gen, *shape).to(dtype), (2 * _randn(gen, *shape)).to(dtype)
    st = {"c": c, "post": 1 + 0.1 * _randn(gen, h) if c["post"] else None,
          "pre": 1 + 0.1 * _randn(gen, h) if c["pre"] else None, "gate": None, "y": y}
    if c["gate"] != "none":
        st["gate"] = 0.5 * _randn(gen, *((h,) if c["gate"] == "vector" else (c["b"], h)))
    if c["op"] == "residual_norm":
        st["x"] = x
    else:  # any finite r will do for the gradients: the forward's is of the size of x + y
        st["r"] = x
        st["dr"] = _randn(gen, *shape).to(dtype)
        st["du"] = _randn(gen, *shape).to(dtype) if c["pre"] else None
    return st


# ----------------------------------------------------------------------------- plain forms

def _act(c, z):
    if c["act"] == "silu":
        return z / (1 + torch.exp(-z))
    if c["act"] == "gelu_tanh":
        return 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z * z * z)))
    return 0.5 * z * (1 + torch.erf(z * math.sqrt(0.5)))


def _act_slope(c, z):
    if c["act"] == "silu":
        sig = 1 / (1 + torch.exp(-z))
        return sig * (1 + z * (1 - sig))
    if c["act"] == "gelu_tanh":
        k = math.sqrt(2 / math.pi)
        th = torch.tanh(k * (z + 0.044715 * z * z * z))
        return 0.5 * (1 + th) + 0.5 * z * (1 - th * th) * k * (1 + 3 * 0.044715 * z * z)
    return 0.5 * (1 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(-0.5 * z * z) / math.sqrt(2 * math.pi)


def _plain_gated(st):
    c = st["c"]
    z = st["X"].float() @ st["A"].float()
    gate, up = _shards(c, z)
    y = _act(c, gate) * up
    o = (y @ st["B"].float()).to(torch.bfloat16)
    return (o, z.to(torch.bfloat16), y.to(torch.bfloat16)) if c["save"] else o


def _plain_gated_grad(st):
    c = st["c"]
    gate, up = _shards(c, st["Z"].float())
    g = st["G"].float()
    dy = g @ st["B"].float().T
    dz = _join(c, dy * up * _act_slope(c, gate), dy * _act(c, gate))
    return tuple(v.to(torch.bfloat16) for v in (dz @ st["A"].float().T, st["X"].float().T @ dz, st["Y"].float().T @ g))


def _root(x):
    return torch.rsqrt((x * x).mean(-1, keepdim=True) + _EPS)


def _plain_gate(st):
    g = st["gate"]
    return g if g is None or g.dim() == 1 else g[:, None]


def _plain_norm(st):
    c, gate = st["c"], _plain_gate(st)
    p = st["y"].float()
    if st["post"] is not None:
        p = p * _root(p) * st["post"]
    if gate is not None:
        p = p * gate
    r = c["alpha"] * st["x"].float() + p
    dtype = st["x"].dtype
    return (r.to(dtype),) if st["pre"] is None else (r.to(dtype), (r * _root(r) * st["pre"]).to(dtype))


def _plain_norm_back(x, gamma, dy):
    """dx and dgamma of rmsnorm(x) gamma."""
    r = _root(x)
    xhat, g = x * r, dy * gamma
    return r * (g - xhat * (g * xhat).mean(-1, keepdim=True)), (dy * xhat).double().sum((0, 1)).float()


def _plain_norm_grad(st):
    c, gate = st["c"], _plain_gate(st)
    y, out = st["y"].float(), {}
    g = st["dr"].float()
    if st["pre"] is not None:
        more, out["dpre"] = _plain_norm_back(st["r"].float(), st["pre"], st["du"].float())
        g = g + more
    if gate is not None:
        p = y if st["post"] is None else y * _root(y) * st["post"]
        out["dgate"] = (g * p).double().sum((0, 1) if st["gate"].dim() == 1 else 1).float()
    dy = g if gate is None else g * gate
    if st["post"] is not None:
        dy, out["dpost"] = _plain_norm_back(y, st["post"], dy)
    out["dx"], out["dy"] = (c["alpha"] * g).to(st["y"].dtype), dy.to(st["y"].dtype)
    return out


_PLAIN = {"gated": _plain_gated, "gated_grad": _plain_gated_grad, "residual_norm": _plain_norm,
          "residual_norm_grad": _plain_norm_grad}


# ----------------------------------------------------------------------------- the framework's calls

def _run_own(st):
    import tensor_transformer_mlp_gb300 as tp

    c = st["c"]
    if c["op"] == "gated":
        o, z, y = tp.gated_forward(st["X"], st["A"], st["B"], c["t"], c["act"], save=c["save"])
        return (o, z, y) if c["save"] else o
    if c["op"] == "gated_grad":
        return tp.gated_backward(st["X"], st["A"], st["B"], st["G"], st["Z"], st["Y"], c["t"], c["act"],
                                 wgrad="operand")
    if c["op"] == "residual_norm":
        r, u = tp.residual_norm(st["x"], st["y"], gamma_post=st["post"], gate=st["gate"], gamma_pre=st["pre"],
                                alpha=c["alpha"], eps=_EPS)
        return (r,) if u is None else (r, u)
    dx, dy, dpost, dgate, dpre = tp.residual_norm_backward(st["y"], st["r"], st["dr"], st["du"], gamma_post=st["post"],
                                                           gate=st["gate"], gamma_pre=st["pre"], alpha=c["alpha"],
                                                           eps=_EPS)
    out = {"dx": dx, "dy": dy, "dpost": dpost, "dgate": dgate, "dpre": dpre}
    return {k: v for k, v in out.items() if v is not None}


def run(state):
    return _run_own(state) if own else _PLAIN[state["c"]["op"]](state)


# ----------------------------------------------------------------------------- work and exact values

def work(case):
    c = case
    if c["op"].startswith("gated"):
        n, d, m = c["n"], c["d"], c["m"]
        if c["op"] == "gated":  # three products of n d m
            return {"bytes": 2 * (2 * n * d + 3 * d * m + (3 * n * m if c["save"] else 0)), "flops": 6.0 * n * d * m}
        return {"bytes": 2 * (3 * n * d + 3 * n * m + 6 * d * m), "flops": 12.0 * n * d * m}
    size, values = (2 if c["dtype"] == BF16 else 4), c["b"] * c["s"] * c["h"]
    gate = {"none": 0, "vector": c["h"], "sequence": c["b"] * c["h"]}[c["gate"]]
    params = 4 * (gate + c["h"] * (c["post"] + c["pre"]))
    if c["op"] == "residual_norm":
        return {"bytes": values * size * (3 + c["pre"]) + params, "flops": 8 * values}
    return {"bytes": values * size * (4 if c["post"] or c["gate"] != "none" else 3) + values * size * 2 * c["pre"]
            + 2 * params, "flops": 20 * values}


def _exact_act(c, z):
    if c["act"] == "silu":
        return z * torch.sigmoid(z)
    if c["act"] == "gelu_tanh":  # (1 + tanh w) / 2 = sigmoid(2 w)
        return z * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3))
    return z * torch.special.ndtr(z)


def _exact_gated(st):
    c = st["c"]
    x, mt = st["X"].double(), c["m"] // c["t"]
    o, z, y = 0.0, [], []
    for i in range(c["t"]):  # shard by shard
        for part in range(2):
            lo = (2 * i + part) * mt
            z.append(x @ st["A"][:, lo:lo + mt].double())
        y.append(_exact_act(c, z[-2]) * z[-1])
        o = o + y[-1] @ st["B"][i * mt:(i + 1) * mt].double()
    return (o, torch.cat(z, 1), torch.cat(y, 1)) if c["save"] else o


def _exact_gated_grad(st):
    c = st["c"]
    x, g, mt = st["X"].double(), st["G"].double(), c["m"] // c["t"]
    dx, da = 0.0, []
    for i in range(c["t"]):
        lo = 2 * i * mt
        gate = st["Z"][:, lo:lo + mt].double().requires_grad_()
        up = st["Z"][:, lo + mt:lo + 2 * mt].double().requires_grad_()
        dy = g @ st["B"][i * mt:(i + 1) * mt].double().T
        for k, dz in enumerate(torch.autograd.grad(_exact_act(c, gate) * up, (gate, up), dy)):
            dx = dx + dz @ st["A"][:, lo + k * mt:lo + (k + 1) * mt].double().T
            da.append(x.T @ dz)
    return dx, torch.cat(da, 1), st["Y"].double().T @ g


def _exact_rms(v, gamma):
    return v / torch.sqrt(v.square().sum(-1, keepdim=True) / v.shape[-1] + _EPS) * gamma


def _exact_norm(st):
    c = st["c"]
    p = st["y"].double()
    if st["post"] is not None:
        p = _exact_rms(p, st["post"].double())
    if st["gate"] is not None:
        p = torch.einsum("bsh,bh->bsh", p, st["gate"].double().expand(c["b"], c["h"]))
    r = st["x"].double() * c["alpha"] + p
    return (r,) if st["pre"] is None else (r, _exact_rms(r, st["pre"].double()))


def _exact_norm_grad(st):
    """By differentiation: of u's share in r, and of what y adds to r."""
    c, out = st["c"], {}
    g = st["dr"].double()
    if st["pre"] is not None:
        r, gamma = st["r"].double().requires_grad_(), st["pre"].double().requires_grad_()
        more, out["dpre"] = torch.autograd.grad(_exact_rms(r, gamma), (r, gamma), st["du"].double())
        g = g + more
    out["dx"] = g * c["alpha"]
    leaves = {"dy": st["y"].double().requires_grad_()}
    p = leaves["dy"]
    if st["post"] is not None:
        leaves["dpost"] = st["post"].double().requires_grad_()
        p = _exact_rms(p, leaves["dpost"])
    if st["gate"] is not None:
        leaves["dgate"] = st["gate"].double().requires_grad_()
        p = torch.einsum("bsh,bh->bsh", p, leaves["dgate"].expand(c["b"], c["h"]))
    out.update(zip(leaves, torch.autograd.grad(p, tuple(leaves.values()), g)))
    return out


_EXACT = {"gated": _exact_gated, "gated_grad": _exact_gated_grad, "residual_norm": _exact_norm,
          "residual_norm_grad": _exact_norm_grad}


def exact(case, seed):
    return _EXACT[case["op"]](prepare(case, seed))
