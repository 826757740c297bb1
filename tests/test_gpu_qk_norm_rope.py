"""GPU parity of the per-head norm with rotation and its backward against the float64 oracle.

Tolerances, element by element: outputs are fp32 arithmetic rounded once to the tensor's type, so u |y| with u = 2^-8
(bf16) or 2^-23 (fp32: the rounding of the result and of its last operation), plus fp32 arithmetic on values of the
head's size: a dozen operations and a sum over head_dim of 2^-24 each, 2^-18 of the head's largest term."""
import numpy as np
import pytest
import torch

import tensor_transformer_mlp_gb300 as tp
from oracle import qk_norm_rope as oqr

pytestmark = pytest.mark.gpu

U = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -23}
EPS = 1e-5


def _np(t):
    return t.double().cpu().numpy()


def _hold(name, got, ref, tol):
    got = _np(got)
    assert got.shape == ref.shape
    over = np.abs(got - ref) - tol
    assert np.isfinite(got).all(), name
    at = np.unravel_index(np.argmax(over), over.shape)
    assert over[at] <= 0, f"{name}{list(map(int, at))}: {got[at]} for {ref[at]}, tolerance {tol[at]}"


def _inputs(seed, b, s, heads, kv, hd, rot, dtype, packed=False, table=500):
    gen = torch.Generator("cuda").manual_seed(seed)
    rand = lambda *shape: torch.randn(*shape, generator=gen, device="cuda").to(dtype)  # noqa: E731
    if packed:
        m = rand(b, s, heads, 3, hd)
        q, k = m[:, :, :, 0], m[:, :, :, 1]
    else:
        m = rand(b, s, (heads + 2 * kv) * hd)
        q, k = m[..., :heads * hd].unflatten(-1, (heads, hd)), m[..., heads * hd:(heads + kv) * hd].unflatten(-1, (kv, hd))
    gq, gk = (1 + 0.3 * torch.randn(hd, generator=gen, device="cuda") for _ in range(2))
    cos, sin = tp.rope_tables(table, rot, device="cuda")
    pos = torch.randint(0, table, (b, s), generator=gen, device="cuda", dtype=torch.int32)
    return q, k, gq, gk, cos, sin, pos, rand(b, s, heads, hd), rand(b, s, kv, hd)


def _check(inp, style, positions, eps=EPS):
    q, k, gq, gk, cos, sin, pos, dyq, dyk = inp
    b, s, _, hd = q.shape
    p = pos if positions else None
    outs = tp.qk_norm_rope(q, k, gq, gk, cos, sin, eps=eps, positions=p, style=style)
    dq, dk, dgq, dgk = tp.qk_norm_rope_backward(q, k, gq, gk, cos, sin, dyq, dyk, eps=eps, positions=p, style=style)
    torch.cuda.synchronize()
    at = _np(pos).astype(int).reshape(-1) if positions else np.tile(np.arange(s), b)
    c, sn = cos.cpu().numpy(), sin.cpu().numpy()
    for name, x, g, y, dy, dx, dg in (("q", q, gq, outs[0], dyq, dq, dgq), ("k", k, gk, outs[1], dyk, dk, dgk)):
        u = U[x.dtype]
        x, dy = (_np(t).reshape(b * s, -1, hd) for t in (x, dy))
        ref = oqr.forward(x, _np(g), eps, c, sn, at, style)
        _hold(name, y.reshape(ref.shape), ref, u * np.abs(ref) + 2.0 ** -18 * np.abs(ref).max(-1, keepdims=True) + 1e-30)
        rx, rg = oqr.backward(x, _np(g), eps, c, sn, at, style, dy)
        r = 1 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
        size = r * np.abs(dy).max(-1, keepdims=True) * np.abs(_np(g)).max() * 4   # dx's terms
        _hold("d" + name, dx.reshape(rx.shape), rx, u * np.abs(rx) + 2.0 ** -18 * size + 1e-30)
        terms = np.abs(dy).max() * np.abs(x * r).sum((0, 1)) * 2
        _hold("dgamma_" + name, dg, rg, 2.0 ** -18 * terms + 1e-30)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("style", ["half", "interleaved"])
@pytest.mark.parametrize("hd,rot", [(8, 8), (8, 2), (16, 16), (40, 20), (64, 64), (64, 32), (72, 36), (80, 40), (80, 80),
                                    (96, 96), (128, 128), (128, 64), (136, 136), (256, 256), (256, 50)])
def test_head_widths(dtype, style, hd, rot):
    _check(_inputs(hd + rot, 2, 19, 4, 2, hd, rot, dtype), style, True)


@pytest.mark.parametrize("b,s", [(1, 1), (4, 1), (1, 33), (3, 129), (2, 400)])
@pytest.mark.parametrize("heads,kv", [(1, 1), (5, 5), (32, 8), (33, 3), (70, 70)])
def test_shapes(b, s, heads, kv):
    _check(_inputs(s + heads, b, s, heads, kv, 32, 32, torch.bfloat16, packed=heads == kv), "half", s % 2 == 1)


def test_many_tokens_sum_their_gains():
    _check(_inputs(1, 3, 1700, 4, 4, 64, 64, torch.float32, packed=True, table=1700), "half", False)
    _check(_inputs(2, 1, 6000, 2, 1, 128, 128, torch.bfloat16, table=6000), "interleaved", False)


def test_large_eps_and_zero_rows():
    inp = _inputs(4, 1, 20, 2, 2, 64, 64, torch.float32)
    inp[0][0, 3] = 0
    _check(inp, "half", True, eps=0.5)


@pytest.mark.parametrize("eps", [1e-12, 1e-30])
def test_tiny_eps_and_zero_rows(eps):
    # 1 / sqrt(eps) is 1e15 there, and its cube is past fp32
    inp = _inputs(9, 1, 20, 2, 2, 64, 64, torch.float32)
    inp[0][0, 3] = 0
    inp[1][0, 5] = 0
    _check(inp, "interleaved", True, eps=eps)


def test_in_place_and_into_views():
    q, k, gq, gk, cos, sin, pos, dyq, dyk = _inputs(5, 2, 31, 6, 6, 40, 20, torch.bfloat16, packed=True)
    want = tp.qk_norm_rope(q, k, gq, gk, cos, sin, positions=pos)
    grads = tp.qk_norm_rope_backward(q, k, gq, gk, cos, sin, dyq, dyk, positions=pos)
    tp.qk_norm_rope_backward(q, k, gq, gk, cos, sin, dyq, dyk, positions=pos, dq=dyq, dk=dyk)
    assert torch.equal(grads[0], dyq) and torch.equal(grads[1], dyk)
    rest = q._base[:, :, :, 2].clone() if q._base is not None else None
    tp.qk_norm_rope(q, k, gq, gk, cos, sin, positions=pos, q_out=q, k_out=k)
    assert torch.equal(q, want[0]) and torch.equal(k, want[1])
    if rest is not None:
        assert torch.equal(q._base[:, :, :, 2], rest)        # the values in between


def test_padding_and_positions_behind_the_table():
    q, k, gq, gk, cos, sin, pos, dyq, dyk = _inputs(6, 1, 12, 2, 1, 64, 32, torch.bfloat16, table=50)
    pos[0, 4], pos[0, 5], pos[0, 7] = -1, -2 ** 31, 50
    q[0, 4] = float("nan")
    dyq[0, 5] = float("inf")
    y = tp.qk_norm_rope(q, k, gq, gk, cos, sin, positions=pos)
    g = tp.qk_norm_rope_backward(q, k, gq, gk, cos, sin, dyq, dyk, positions=pos)
    for t in (*y, g[0], g[1]):
        assert torch.count_nonzero(t[0, 4:6]) == 0
        assert torch.isfinite(t[0, [0, 1, 2, 3, 6, 8, 9, 10, 11]]).all()
    assert torch.isnan(y[0][0, 7, :, :32]).all() and torch.isfinite(y[0][0, 7, :, 32:]).all()
    assert torch.isnan(g[2]).any()                            # the loss of such a row is no number
    pos[0, 7] = 49
    g = tp.qk_norm_rope_backward(q, k, gq, gk, cos, sin, dyq, dyk, positions=pos)
    assert torch.isfinite(g[2]).all() and torch.isfinite(g[3]).all()


def test_empty_batch():
    q = torch.empty(0, 5, 2, 64, dtype=torch.bfloat16, device="cuda")
    g = torch.ones(64, device="cuda")
    cos, sin = tp.rope_tables(8, 64, device="cuda")
    y, _ = tp.qk_norm_rope(q, q, g, g, cos, sin)
    dq, dk, dgq, dgk = tp.qk_norm_rope_backward(q, q, g, g, cos, sin, q, q)
    assert y.shape == q.shape and torch.count_nonzero(dgq) == 0 and torch.count_nonzero(dgk) == 0


def test_far_positions_keep_their_phase():
    # a table of 2^18 positions: the fp32 entries are the rounded cosines of the 64-bit angles
    cos, sin = tp.rope_tables(1 << 18, 128, theta=5e5, device="cuda")
    pos = np.array([0, 1, 131071, 262143])
    ang = pos[:, None].astype(np.longdouble) * np.longdouble(5e5) ** (-np.arange(0, 128, 2, dtype=np.longdouble) / 128)
    assert np.abs(cos[pos].cpu().numpy() - np.cos(ang)).max() < 2.0 ** -24 and np.abs(sin[pos].cpu().numpy() - np.sin(ang)).max() < 2.0 ** -24


def test_graph_and_stream_and_bits():
    q, k, gq, gk, cos, sin, pos, dyq, dyk = _inputs(8, 2, 300, 8, 2, 128, 128, torch.bfloat16)

    def step(stream=None):
        return (tp.qk_norm_rope(q, k, gq, gk, cos, sin, positions=pos, stream=stream)
                + tp.qk_norm_rope_backward(q, k, gq, gk, cos, sin, dyq, dyk, positions=pos, stream=stream))

    want = [t.clone() for t in step()]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = step(side)
    torch.cuda.current_stream().wait_stream(side)
    for a, b in zip(want, got):
        assert torch.equal(a, b)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step()
    for t in held:
        t.zero_()
    graph.replay()
    torch.cuda.synchronize()
    for a, b in zip(want, held):
        assert torch.equal(a, b)


def test_offsets_past_32_bits():
    s, ld = 36000, 65536
    big = torch.zeros(s, ld, dtype=torch.bfloat16, device="cuda")
    gen = torch.Generator("cuda").manual_seed(3)
    big[:, :256] = torch.randn(s, 256, generator=gen, device="cuda").bfloat16()
    q, k = big[:, :128].view(1, s, 2, 64), big[:, 128:256].view(1, s, 2, 64)
    yq = big[:, ld - 128:].view(1, s, 2, 64)
    g = torch.ones(64, device="cuda")
    cos, sin = tp.rope_tables(s, 64, device="cuda")
    tp.qk_norm_rope(q, k, g, g, cos, sin, q_out=yq)
    tail = slice(s - 40, s)
    ref = oqr.forward(_np(q[0, tail]), _np(g), EPS, cos.cpu().numpy(), sin.cpu().numpy(), np.arange(s - 40, s), "half")
    _hold("q", yq[0, tail], ref, U[torch.bfloat16] * np.abs(ref) + 2.0 ** -18 * np.abs(ref).max(-1, keepdims=True))
