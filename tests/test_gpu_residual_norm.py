"""The norms around a block on the GPU against their float64 oracle.

Tolerances. fp32 sums over h columns are taken by threads of up to 16 columns each and a tree: off by at most 2^-19 of the
sum of magnitudes for any h here (some 30 roundings of 2^-24). Everything behind them is a handful of fp32 operations: a
value is good to E = 2^-18 of the sum of the magnitudes of its terms. bf16 outputs add half a step, 2^-8 of themselves. Sums
over tokens run over 1024 partial sums at the most and what a CTA adds one after another; each is off by its number of terms
times 2^-24 of the sum of magnitudes, and independent roundings by their root, of which 8 are allowed: 8 sqrt(n) 2^-24."""
import itertools

import numpy as np
import pytest
import torch

import tensor_transformer_mlp_gb300 as tp
from oracle import residual_norm as orn

from helpers import host

pytestmark = pytest.mark.gpu

E = 2.0 ** -18
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
EPS = 1e-5


def case(b, s, h, dtype, form=(True, True, True), seed=0):
    gen = torch.Generator("cuda").manual_seed(seed)

    def draw(*shape):
        return torch.randn(*shape, generator=gen, device="cuda")
    c = {k: draw(b, s, h).to(dtype) for k in ("x", "y", "dr", "du")}
    c["post"] = 1 + 0.1 * draw(h) if form[0] else None
    c["gate"] = draw(b, h) if form[1] else None
    c["pre"] = 1 + 0.1 * draw(h) if form[2] else None
    if not form[2]:
        c["du"] = None
    return c


def np64(t):
    return None if t is None else host(t)


def within(name, got, ref, bound):
    got = host(got)
    assert got.shape == ref.shape, name
    assert np.all(np.isfinite(got)), name
    over = np.abs(got - ref) / (bound + 1e-30)
    assert over.size == 0 or over.max() <= 1, (name, over.max(), np.unravel_index(over.argmax(), over.shape))


def check_forward(c, r, u, alpha):
    x, y, post, gate, pre = (np64(c[k]) for k in ("x", "y", "post", "gate", "pre"))
    rr, uu = orn.forward(x, y, post, gate, pre, alpha, EPS)
    half = HALF[c["y"].dtype]
    mag = np.abs(alpha * x) + np.abs(rr - alpha * x)
    within("r", r, rr, half * np.abs(rr) + E * mag)
    if pre is None:
        assert u is None
        return
    root = 1 / np.sqrt((rr * rr).mean(-1, keepdims=True) + EPS)
    # the root is off by E of itself and by what r's slips do to it, at most their own size in the mean
    slip = E * (np.abs(uu) * (1 + np.sqrt((mag * mag).mean(-1, keepdims=True)) * root) + np.abs(pre) * root * mag)
    within("u", u, uu, half * np.abs(uu) + slip)


def magnitudes(c, r, alpha):
    """The sums of magnitudes of g's and dy's terms."""
    y, r, dr, du, post, gate, pre = (np64(v) for v in (c["y"], r, c["dr"], c["du"], c["post"], c["gate"], c["pre"]))
    g = np.zeros_like(y) if dr is None else np.abs(dr)
    if pre is not None:
        root = 1 / np.sqrt((r * r).mean(-1, keepdims=True) + EPS)
        d = np.abs(du * pre)
        g = g + root * (d + np.abs(r * root) * (d * np.abs(r * root)).mean(-1, keepdims=True))
    root = 1 / np.sqrt((y * y).mean(-1, keepdims=True) + EPS) if post is not None else np.ones_like(y[..., :1])
    w = np.ones(y.shape[-1]) if post is None else np.abs(post)
    w = w if gate is None else w * np.abs(gate[:, None])
    dy = w * g
    if post is not None:
        hat = np.abs(y) * root
        dy = root * (dy + hat * (dy * hat).mean(-1, keepdims=True))
    return g, dy, np.abs(y) * root


def check_backward(c, r, got, alpha):
    names = ("dx", "dy", "dpost", "dgate", "dpre")
    want = orn.backward(*(np64(v) for v in (c["y"], r, c["dr"], c["du"], c["post"], c["gate"], c["pre"])), alpha, EPS)
    mg, mdy, hat = magnitudes(c, r, alpha)
    half = HALF[c["y"].dtype]
    n = c["y"].shape[0] * c["y"].shape[1]
    many = 8 * np.sqrt(n) * 2.0 ** -24 + E
    gate = None if c["gate"] is None else np64(c["gate"])
    bound = {"dx": half * np.abs(want["dx"]) + E * abs(alpha) * mg, "dy": half * np.abs(want["dy"]) + E * mdy}
    if c["post"] is not None:
        bound["dpost"] = many * (mg * hat * (1 if gate is None else np.abs(gate[:, None]))).sum((0, 1))
    if gate is not None:
        bound["dgate"] = many * (mg * hat).sum(1) * (1 if c["post"] is None else np.abs(np64(c["post"])))
    if c["pre"] is not None:
        rn = np64(r)
        bound["dpre"] = many * np.abs(np64(c["du"]) * rn / np.sqrt((rn * rn).mean(-1, keepdims=True) + EPS)).sum((0, 1))
    for name, t in zip(names, got):
        assert (t is None) == (name not in want), name
        if t is not None:
            within(name, t, want[name], bound[name])


def run(c, alpha=1.0, check=True, **kw):
    gains = dict(gamma_post=c["post"], gate=c["gate"], gamma_pre=c["pre"], alpha=alpha, eps=EPS)
    r, u = tp.residual_norm(c["x"], c["y"], **gains, **kw)
    got = tp.residual_norm_backward(c["y"], r if c["pre"] is not None else None, c["dr"], c["du"], **gains, **kw)
    if check:
        torch.cuda.synchronize()
        tp.tpmlp_device_status()
        check_forward(c, r, u, alpha)
        check_backward(c, r, got, alpha)
    return r, u, got


# every kernel: lane groups of 4 to 32 lanes with one and two vectors, CTAs of 128, 256 and 512 threads
WIDTHS = [8, 24, 64, 136, 256, 264, 512, 520, 1024, 1608, 2048, 2056, 4096, 5000, 8192]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("h", WIDTHS)
def test_widths(h, dtype):
    run(case(3, 37, h, dtype, seed=h), alpha=0.75)


@pytest.mark.parametrize("form", list(itertools.product([False, True], repeat=3)))
@pytest.mark.parametrize("h", [72, 776])
def test_forms(form, h):
    run(case(2, 50, h, torch.bfloat16, form), alpha=1.5)
    run(case(2, 50, h, torch.float32, form))


@pytest.mark.parametrize("h", [64, 320, 1000, 4096])
@pytest.mark.parametrize("b,s", [(1, 1), (5, 1), (1, 3), (700, 1), (300, 3), (7, 151), (2, 1111), (40, 100), (1, 5000)])
def test_how_sequences_fall_on_ctas(b, s, h):
    # sequences within a CTA's rows, across CTAs, CTAs with several sequences, more rows than CTAs and fewer
    run(case(b, s, h, torch.bfloat16, seed=b + s))


def test_learned_gate():
    # [h]: one gate for all tokens, whatever their shape
    c = case(1, 96, 520, torch.float32)
    r, u, got = run(c)
    flat = dict(gamma_post=c["post"], gate=c["gate"][0], gamma_pre=c["pre"])
    r2, u2 = tp.residual_norm(c["x"].view(4, 24, 520), c["y"].view(4, 24, 520), **flat)
    assert torch.equal(r.view_as(r2), r2) and torch.equal(u.view_as(u2), u2)
    got2 = tp.residual_norm_backward(*(v.view(96, 520) for v in (c["y"], r, c["dr"], c["du"])), **flat)
    assert got2[3].shape == (520,)
    for a, b in zip(got, got2):
        assert torch.equal(a.reshape(-1), b.reshape(-1))


@pytest.mark.parametrize("h", [128, 1024])
def test_no_direct_gradient(h):
    c = case(2, 30, h, torch.bfloat16)
    c["dr"] = None
    run(c)


@pytest.mark.parametrize("h", [128, 1024])
def test_y_is_not_needed_without_norm_and_gate(h):
    c = case(2, 30, h, torch.float32, (False, False, True))
    r, _, want = run(c)
    got = tp.residual_norm_backward(None, r, c["dr"], c["du"], gamma_pre=c["pre"], eps=EPS)
    assert torch.equal(want[0], got[0]) and torch.equal(want[1], got[1]) and torch.equal(want[4], got[4])


@pytest.mark.parametrize("h", [256, 2048])
def test_in_place(h):
    c = case(2, 200, h, torch.bfloat16)
    r, u, want = run(c)
    gains = dict(gamma_post=c["post"], gate=c["gate"], gamma_pre=c["pre"], eps=EPS)
    for k, o in (("x", "y"), ("y", "x")):
        a, b = c[k].clone(), c[o].clone()
        ins = {k: a, o: b}
        tp.residual_norm(ins["x"], ins["y"], **gains, r=a, u=b)
        assert torch.equal(a, r) and torch.equal(b, u)
    for i, j in itertools.permutations(range(4), 2):
        ins = [v.clone() for v in (c["y"], r, c["dr"], c["du"])]
        got = tp.residual_norm_backward(*ins, **gains, dx=ins[i], dy=ins[j])
        assert got[0] is ins[i] and got[1] is ins[j]
        for a, b in zip(want, got):
            assert torch.equal(a, b)


@pytest.mark.parametrize("h", [256, 4096])
def test_what_a_row_holds_stays_in_it(h):
    c = case(2, 60, h, torch.bfloat16)
    r, u, want = run(c)
    d = {k: v.clone() for k, v in c.items()}
    d["x"][1, 17], d["y"][0, 3], d["dr"][1, 18] = float("inf"), float("nan"), float("nan")
    r2, u2, got = run(d, check=False)
    keep = torch.ones(2, 60, dtype=torch.bool, device="cuda")
    keep[1, 17] = keep[0, 3] = False
    assert torch.equal(r[keep], r2[keep]) and torch.equal(u[keep], u2[keep])
    keep[1, 18] = False
    assert torch.equal(want[0][keep], got[0][keep]) and torch.equal(want[1][keep], got[1][keep])
    assert torch.isnan(got[0][1, 18]).any() and torch.isnan(got[3]).any()


def test_rows_of_zeros_and_large_values():
    c = case(1, 40, 1024, torch.float32)
    c["y"][0, 5], c["x"][0, 5] = 0, 0                  # eps alone under the root
    c["y"][0, 6] *= 1e15
    c["x"][0, 7] *= 1e-15
    r, u = tp.residual_norm(c["x"], c["y"], c["post"], c["gate"][0], c["pre"], eps=EPS)
    assert not r[0, 5].any() and not u[0, 5].any()
    check_forward(c, r, u, 1.0)


def test_residual_that_cancels():
    # r is a small difference of x and the block's share: its norm is taken from r itself
    c = case(1, 30, 1024, torch.float32, (False, False, True))
    c["x"] = -c["y"] * (1 + 1e-3 * torch.randn_like(c["y"]))
    run(c)


def test_no_tokens():
    for b, s in ((0, 4), (3, 0)):
        c = case(b, s, 64, torch.bfloat16)
        r, u, got = run(c, check=False)
        assert r.shape == u.shape == (b, s, 64) and got[3].shape == (b, 64)
        assert not any(got[k].any() for k in (2, 3, 4))


@pytest.mark.parametrize("h", [256, 4096])
def test_on_another_stream_from_a_graph_and_again(h):
    c = case(3, 333, h, torch.bfloat16)
    r, u, want = run(c)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for _ in range(3):                                  # the same bits every time
        r2, u2, got = run(c, check=False, stream=side)
        side.synchronize()
        for a, b in zip((r, u) + want, (r2, u2) + got):
            assert torch.equal(a, b)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cap = run(c, check=False)
    for _ in range(2):
        for k in ("x", "y", "dr", "du"):
            c[k].copy_(c[k].flip(1))
        graph.replay()
    torch.cuda.synchronize()
    for a, b in zip((r, u) + want, cap[:2] + cap[2]):
        assert torch.equal(a, b)
    tp.tpmlp_device_status()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("h", [256, 520, 2048])
def test_gradients_of_rows_of_zeros_and_large_values(h, dtype, monkeypatch):
    # roots from 1e15 (an eps of 1e-30 alone) to 1e-15, whose cubes fp32 does not hold
    monkeypatch.setitem(globals(), "EPS", 1e-30)
    for dr in (True, False):
        c = case(2, 40, h, dtype)
        c["x"][0, 5], c["y"][0, 5] = 0, 0
        c["x"][0, 6:8] *= 1e15
        c["y"][0, 8:10] *= 1e15
        c["x"][1, 7] *= 1e15
        c["y"][1, 7] *= 1e15
        if not dr:
            c["dr"] = None
        run(c)


def test_backward_on_two_streams_at_once():
    cs = [case(3, 700, 2048, torch.bfloat16, seed=k) for k in range(2)]
    want = [run(c)[2] for c in cs]
    streams = [torch.cuda.Stream() for _ in cs]
    torch.cuda.synchronize()
    got = [None, None]
    for _ in range(4):
        for k, (c, s) in enumerate(zip(cs, streams)):
            got[k] = run(c, check=False, stream=s)[2]
    torch.cuda.synchronize()
    for w, g in zip(want, got):
        assert all(torch.equal(a, b) for a, b in zip(w, g))
    tp.tpmlp_device_status()


# from 4800 rows on in sequences of 64 tokens and more: a warp takes a row of 257 to 512 columns (bf16: 1024)
@pytest.mark.parametrize("h,dtype", [(264, torch.float32), (512, torch.float32), (264, torch.bfloat16), (512, torch.bfloat16),
                                     (520, torch.bfloat16), (768, torch.bfloat16), (776, torch.bfloat16), (1024, torch.bfloat16)])
@pytest.mark.parametrize("b,s", [(1, 4800), (75, 64), (53, 100), (3, 1733), (7, 1000)])
def test_rows_of_a_warp(b, s, h, dtype):
    run(case(b, s, h, dtype), alpha=0.75)


@pytest.mark.parametrize("form", list(itertools.product([False, True], repeat=3)))
def test_rows_of_a_warp_in_every_form(form):
    run(case(2, 2500, 904, torch.bfloat16, form), alpha=-1.5)
    run(case(2, 2500, 312, torch.float32, form), alpha=-1.5)


def test_rows_of_a_warp_in_place_and_alone():
    c = case(2, 2600, 1000, torch.bfloat16)
    r, u, want = run(c)
    gains = dict(gamma_post=c["post"], gate=c["gate"], gamma_pre=c["pre"], eps=EPS)
    for first, second in itertools.permutations(("y", "r", "dr", "du"), 2):
        t = {k: (r if k == "r" else c[k]).clone() for k in ("y", "r", "dr", "du")}
        got = tp.residual_norm_backward(t["y"], t["r"], t["dr"], t["du"], **gains, dx=t[first], dy=t[second])
        assert got[0] is t[first] and got[1] is t[second]
        assert all(torch.equal(a, b) for a, b in zip(want, got))
    bad = {k: v.clone() for k, v in (("y", c["y"]), ("r", r), ("dr", c["dr"]), ("du", c["du"]))}
    bad["dr"][1, 18, 3] = float("nan")
    got = tp.residual_norm_backward(*bad.values(), **gains)
    keep = torch.ones(2, 2600, dtype=torch.bool, device="cuda")
    keep[1, 18] = False
    assert torch.equal(want[0][keep], got[0][keep]) and torch.equal(want[1][keep], got[1][keep])
    assert torch.isnan(got[0][1, 18]).any() and torch.isnan(got[3]).any()
    no_dr = tp.residual_norm_backward(c["y"], r, None, c["du"], **gains)
    check_backward({**c, "dr": None}, r, no_dr, 1.0)


@pytest.mark.parametrize("form", list(itertools.product([False, True], repeat=3)))
@pytest.mark.parametrize("h", [4104, 5120, 8192])
def test_wide_fp32_rows(h, form):
    run(case(3, 167, h, torch.float32, form), alpha=0.75)


def test_wide_fp32_rows_in_place():
    c = case(2, 200, 6152, torch.float32)
    r, u, want = run(c)
    gains = dict(gamma_post=c["post"], gate=c["gate"], gamma_pre=c["pre"], eps=EPS)
    for first, second in itertools.permutations(range(4), 2):
        ins = [v.clone() for v in (c["y"], r, c["dr"], c["du"])]
        got = tp.residual_norm_backward(*ins, **gains, dx=ins[first], dy=ins[second])
        assert all(torch.equal(a, b) for a, b in zip(want, got))
