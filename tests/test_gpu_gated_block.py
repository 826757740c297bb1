"""The gated feed-forward block between its norms, as a transformer layer runs it, forward and backward, against the same
layer in 64 bits by automatic differentiation:

    r0, u0 = residual_norm(x, a, gate_a, gains)      (a: the attention's output)
    f      = gated_forward(u0)
    r1, u1 = residual_norm(r0, f, gate_f, gains)

Tolerance: relative 2-norm of each result. A value rounded to bf16 is off by 2^-8 / sqrt(3) of itself at most in the mean
square; at most 8 rounded tensors stand between an input and a result (u0, Z, Y, f, r0, D, du0, and the result), the norms and
products pass a relative error on, and the gate's product adds two: sqrt(8 + 2) 2^-8 / sqrt(3) = 0.0071, and twice that for
what passes both parts of a sum that partly cancel."""
import math
import os
import subprocess
import sys

import pytest
import torch

import tensor_transformer_mlp_gb300 as tp

pytestmark = pytest.mark.gpu

TOL = 2 * math.sqrt(10) * 2.0 ** -8 / math.sqrt(3)
EPS, ALPHA = 1e-5, 1.25


def rms(x, gamma):
    return x / torch.sqrt((x * x).mean(-1, keepdim=True) + EPS) * gamma


def layer64(p, t):
    b, s, h = p["x"].shape
    r0 = p["x"] + p["gate_a"][:, None] * rms(p["a"], p["post_a"])
    u0 = rms(r0, p["pre_f"]).view(b * s, h)
    z = (u0 @ p["A"]).view(b * s, t, 2, -1)
    y = (torch.nn.functional.silu(z[:, :, 0]) * z[:, :, 1]).reshape(b * s, -1)
    f = (y @ p["B"]).view(b, s, h)
    r1 = ALPHA * r0 + p["gate_f"][:, None] * rms(f, p["post_f"])
    return r1, rms(r1, p["pre_n"])


def layer(p, t, dr1, du1):
    b, s, h = p["x"].shape
    first = dict(gamma_post=p["post_a"], gate=p["gate_a"], gamma_pre=p["pre_f"], eps=EPS)
    second = dict(gamma_post=p["post_f"], gate=p["gate_f"], gamma_pre=p["pre_n"], alpha=ALPHA, eps=EPS)
    r0, u0 = tp.residual_norm(p["x"], p["a"], **first)
    u0 = u0.view(b * s, h)
    f, z, y = tp.gated_forward(u0, p["A"], p["B"], t)
    f = f.view(b, s, h)
    r1, u1 = tp.residual_norm(r0, f, **second)
    g = {}
    dr0, df, g["post_f"], g["gate_f"], g["pre_n"] = tp.residual_norm_backward(f, r1, dr1, du1, **second)
    du0, g["A"], g["B"] = tp.gated_backward(u0, p["A"], p["B"], df.view(b * s, h), z, y, t)
    g["x"], g["a"], g["post_a"], g["gate_a"], g["pre_f"] = tp.residual_norm_backward(p["a"], r0, dr0, du0.view(b, s, h), **first)
    return r1, u1, g


def make(b, s, h, m, seed=0):
    gen = torch.Generator("cuda").manual_seed(seed)

    def draw(*shape):
        return torch.randn(*shape, generator=gen, device="cuda")
    p = {k: draw(b, s, h).bfloat16() for k in ("x", "a")}
    p["A"], p["B"] = (h ** -0.5 * draw(h, 2 * m)).bfloat16(), (m ** -0.5 * draw(m, h)).bfloat16()
    p.update({k: 1 + 0.1 * draw(h) for k in ("post_a", "pre_f", "post_f", "pre_n")})
    p.update({k: 0.5 + 0.2 * draw(b, h) for k in ("gate_a", "gate_f")})
    return p, draw(b, s, h).bfloat16(), draw(b, s, h).bfloat16()


# single tokens of five sequences; a ragged batch; more tokens than a tile of every kernel
@pytest.mark.parametrize("shape", [(5, 1, 512, 1024, 2), (3, 77, 264, 720, 3), (2, 300, 1024, 2048, 4)])
def test_layer(shape):
    b, s, h, m, t = shape
    p, dr1, du1 = make(b, s, h, m, seed=s)
    r1, u1, grads = layer(p, t, dr1, du1)
    torch.cuda.synchronize()
    tp.tpmlp_device_status()
    q = {k: v.double().requires_grad_() for k, v in p.items()}
    R, V = layer64(q, t)
    want = torch.autograd.grad([R, V], list(q.values()), [dr1.double(), du1.double()])
    for name, got, ref in [("r1", r1, R), ("u1", u1, V)] + [(k, grads[k], w) for k, w in zip(q, want)]:
        rel = ((got.double() - ref).norm() / ref.norm()).item()
        assert got.shape == ref.shape and rel <= TOL, (name, rel)


def test_layer_captured_and_replayed():
    p, dr1, du1 = make(2, 70, 256, 512)
    want = layer(p, 2, dr1, du1)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = layer(p, 2, dr1, du1)
    for _ in range(2):
        p["x"].copy_(p["x"].flip(2))                    # there and back
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(want[0], got[0]) and torch.equal(want[1], got[1])
    assert all(torch.equal(want[2][k], got[2][k]) for k in want[2])


COLD = """
import torch
from tests import test_gpu_gated_block as block
import tensor_transformer_mlp_gb300 as tp
p, dr1, du1 = block.make(*{shape})
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    got = block.layer(p, 2, dr1, du1)
graph.replay()
torch.cuda.synchronize()
want = block.layer(p, 2, dr1, du1)
assert torch.equal(want[0], got[0]) and torch.equal(want[1], got[1])
assert all(torch.equal(want[2][k], got[2][k]) for k in want[2])
tp.tpmlp_device_status()
print("same")
"""


@pytest.mark.parametrize("shape", [(3, 1, 512, 1024), (2, 900, 1024, 2048)])
def test_a_process_whose_first_calls_are_captured(shape):
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    out = subprocess.run([sys.executable, "-c", COLD.format(shape=shape)], cwd=root, capture_output=True, text=True, timeout=300)
    assert out.returncode == 0 and out.stdout.strip() == "same", out.stderr[-2000:]


# What the memory of the workspaces and outputs held before must not matter: it is handed out full of NaN.
@pytest.mark.parametrize("wgrad", ["f32", "operand"])
@pytest.mark.parametrize("shape", [(4, 512, 4096, 2), (130, 264, 720, 3), (300, 1024, 2048, 1), (700, 520, 1040, 2), (1111, 1000, 2736, 3)])
def test_memory_full_of_nan(shape, wgrad):
    n, d, m, t = shape
    p, dr, du = make(1, n, d, m)
    gains = dict(gamma_post=p["post_a"], gate=p["gate_a"], gamma_pre=p["pre_f"], eps=EPS)
    X, G = p["x"][0], dr[0]

    def spoil():
        torch.cuda.synchronize()
        held = [torch.full((size,), float("nan"), device="cuda") for size in 8 * [1 << 14] + 8 * [1 << 18] + 8 * [1 << 22]]
        del held

    def steps():
        out = []
        for f in (lambda: tp.gated_forward(X, p["A"], p["B"], t),
                  lambda: tp.gated_backward(X, p["A"], p["B"], G, out[0][1], out[0][2], t, wgrad=wgrad),
                  lambda: tp.residual_norm(p["x"], p["a"], **gains),
                  lambda: tp.residual_norm_backward(p["a"], out[2][0], dr, du, **gains)):
            spoil()
            out.append(f())
        return [v for o in out for v in o]
    first, second = steps(), steps()
    torch.cuda.synchronize()
    tp.tpmlp_device_status()
    for a, b in zip(first, second):
        assert torch.isfinite(a).all() and torch.equal(a, b)
    Z, Y = first[1].double(), first[2].double()
    parts = Z.view(n, t, 2, m // t)
    noise = 2.0 ** -8 / 3 ** 0.5

    def near(a, b, roundings):  # root mean squares: each rounding is off by half a step at most, evenly
        return ((a.double() - b).norm() / b.norm()).item() <= 1.25 * roundings ** 0.5 * noise
    assert near(Z, X.double() @ p["A"].double(), 1)
    assert near(Y, (torch.nn.functional.silu(parts[:, :, 0]) * parts[:, :, 1]).reshape(n, m), 4)
    assert near(first[0], Y @ p["B"].double(), 1)
    assert near(first[5], Y.T @ G.double(), 1)
