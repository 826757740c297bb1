"""The gated feed-forward block on the GPU against its float64 oracle.

Tolerances. u = 2^-8 is half a step of bf16. A product over K values on the tensor core adds K / 16 partial sums in fp32,
each off by at most 2^-22 of the sum of magnitudes: `acc`. Values rounded to bf16 before a product (Y, D) are off by up to
u of themselves, independently: a sum of products with them has a standard deviation of at most u / sqrt(3) times the root
of the sum of squares, and 7 of those are allowed (one value in 10^11). An output rounded to bf16 adds u of itself. tanh.approx
is off by 2^-10.9 of its value; what that does to the gate is added to the deviation."""
import numpy as np
import pytest
import torch

import tensor_transformer_mlp_gb300 as tp
from oracle import gated as og

from helpers import host

pytestmark = pytest.mark.gpu

U = 2.0 ** -8
TANH = 2.0 ** -10.9
ACTS = ["silu", "gelu_tanh", "gelu_erf"]

# (pair kernel, pacing, band): the default choice, 256 x 256 tiles, 256 x 512 tiles, one-SM kernel for the plain products
VARIANTS = {"default": (1, 1, 0), "pair256": (2, 1, 0), "wide": (3, 1, 0), "one_sm": (0, 1, 0), "band5": (3, 1, 5)}


@pytest.fixture(params=list(VARIANTS))
def variant(request):
    tp.tpmlp_set_gemm_variant(*VARIANTS[request.param])
    try:
        yield request.param
    finally:
        tp.tpmlp_set_gemm_variant(1, 1, 0)


def inputs(n, d, m, seed=0, device="cuda"):
    gen = torch.Generator(device).manual_seed(seed)

    def draw(scale, *shape):
        return (scale * torch.randn(*shape, generator=gen, device=device)).bfloat16()
    return draw(1, n, d), draw(d ** -0.5, d, 2 * m), draw(m ** -0.5, m, d), draw(1, n, d)


def acc(k):
    return (k / 16 + 1) * 2.0 ** -22


def within(name, got, ref, bound):
    got = host(got)
    assert got.shape == ref.shape, name
    assert np.all(np.isfinite(got)), name
    over = np.abs(got - ref) / (bound + 1e-30)
    assert over.max() <= 1, (name, over.max(), np.unravel_index(over.argmax(), over.shape))


def tanh_slip(kind, g):
    """What a tanh off by TANH does to (act, act') of gelu_tanh."""
    if kind != "gelu_tanh":
        return 2.0 ** -20 * (1 + np.abs(g)), 2.0 ** -20 * (1 + g * g)
    k = np.sqrt(2 / np.pi)
    th = np.tanh(k * (g + 0.044715 * g ** 3))
    p = np.abs(0.5 * g * k * (1 + 3 * 0.044715 * g * g))
    return 0.5 * np.abs(g * th) * TANH, (2 * p * np.abs(th) + 0.5) * np.abs(th) * TANH


def check_forward(X, A, B, t, kind, O, Z, Y):
    x, a, b = host(X), host(A), host(B)
    d, m = a.shape[0], b.shape[0]
    ref = og.forward(x, a, b, t, kind)
    slip = acc(d) * (np.abs(x) @ np.abs(a))
    if Z is not None:
        within("Z", Z, ref["Z"], U * np.abs(ref["Z"]) + slip)
    gate, up = og.columns(m, t)
    g, u = ref["Z"][:, gate], ref["Z"][:, up]
    act_slip, _ = tanh_slip(kind, g)
    off = 1.2 * slip[:, gate] * np.abs(u) + np.abs(og.act(g, kind)) * slip[:, up] + act_slip * np.abs(u)  # |act'| < 1.2
    within("Y", Y, ref["Y"], U * np.abs(ref["Y"]) + 2 * off)
    dev = np.sqrt(((U / 3 ** 0.5 * ref["Y"]) ** 2 + off ** 2) @ (b * b))
    within("O", O, ref["O"], U * np.abs(ref["O"]) + 7 * dev + acc(m) * (np.abs(ref["Y"]) @ np.abs(b)))


def check_backward(X, A, B, G, Z, Y, t, kind, dX, dA, dB, before=(0.0, 0.0)):
    """dA and dB in fp32 or bf16; `before`: what they held, where the gradients were added to it."""
    x, a, b, g, z, y = (host(v) for v in (X, A, B, G, Z, Y))
    n, d = x.shape
    m = b.shape[0]
    ref = og.backward(x, a, b, g, z, y, t, kind)
    gate, up = og.columns(m, t)
    dy = np.abs(g @ b.T)
    slip_y = acc(d) * (np.abs(g) @ np.abs(b.T))
    s_act, s_grad = tanh_slip(kind, z[:, gate])
    off = np.zeros_like(z)
    off[:, gate] = dy * np.abs(z[:, up]) * s_grad + slip_y * np.abs(z[:, up]) * 1.2
    off[:, up] = dy * s_act + slip_y * (np.abs(z[:, gate]) + 1)
    var = (U / 3 ** 0.5 * ref["D"]) ** 2 + off ** 2
    within("dX", dX, ref["dX"], U * np.abs(ref["dX"]) + 7 * np.sqrt(var @ (a * a).T) + acc(2 * m) * (np.abs(ref["D"]) @ np.abs(a.T)))
    for name, got, dev, mag, old in (("dA", dA, 7 * np.sqrt((x * x).T @ var), np.abs(x).T @ np.abs(ref["D"]), before[0]),
                                     ("dB", dB, 0.0, np.abs(y).T @ np.abs(g), before[1])):
        want = ref[name] + old
        out = U * np.abs(want) if got.dtype == torch.bfloat16 else 2.0 ** -23 * (np.abs(want) + np.abs(old))
        within(name, got, want, out + dev + acc(n) * mag)


def run_and_check(n, d, m, t, kind, wgrad="f32", seed=0):
    X, A, B, G = inputs(n, d, m, seed)
    O, Z, Y = tp.gated_forward(X, A, B, t, kind)
    dX, dA, dB = tp.gated_backward(X, A, B, G, Z, Y, t, kind, wgrad=wgrad)
    torch.cuda.synchronize()
    tp.tpmlp_device_status()
    check_forward(X, A, B, t, kind, O, Z, Y)
    check_backward(X, A, B, G, Z, Y, t, kind, dX, dA, dB)


# Shards of whole column blocks (m / t a multiple of 64), shards that end inside one, shards of 8 columns; rows of less than
# a tile, of more than one, and one.
SHAPES = [(300, 200, 392, 7), (129, 72, 264, 3), (1, 8, 8, 1), (517, 1032, 768, 8), (261, 128, 640, 5), (40, 136, 64, 8),
          (300, 264, 1056, 3)]


@pytest.mark.parametrize("shape", SHAPES)
def test_shapes_on_every_kernel(shape, variant):
    run_and_check(*shape, kind=ACTS[shape[0] % 3], seed=shape[0])


@pytest.mark.parametrize("kind", ACTS)
@pytest.mark.parametrize("wgrad", ["f32", "operand"])
def test_activations_and_gradient_types(kind, wgrad):
    run_and_check(270, 320, 512, 4, kind, wgrad)


@pytest.mark.parametrize("n", [1, 2, 5, 16, 17, 33, 64, 65, 128, 129, 200, 256, 257])
def test_token_counts(n):
    run_and_check(n, 264, 528, 2, "silu", "operand", seed=n)


def test_single_block():
    run_and_check(512, 1024, 4096, 2, "gelu_tanh")


def test_shards_do_not_change_the_products():
    # Columns of A put in shard order give the same Y, O and gradients as one [gate | up] matrix; Z and dA move with them.
    X, A, B, G = inputs(150, 256, 512)
    gate, up = og.columns(512, 4)
    order = torch.from_numpy(np.argsort(np.concatenate([gate, up]))).cuda()
    As = A[:, order].contiguous()
    O1, Z1, Y1 = tp.gated_forward(X, A, B, 1)
    O4, Z4, Y4 = tp.gated_forward(X, As, B, 4)
    assert torch.equal(Y1, Y4) and torch.equal(O1, O4) and torch.equal(Z1[:, order], Z4)
    b1, b4 = tp.gated_backward(X, A, B, G, Z1, Y1, 1), tp.gated_backward(X, As, B, G, Z4, Y4, 4)
    assert torch.equal(b1[1][:, order], b4[1]) and torch.equal(b1[2], b4[2])
    check_backward(X, As, B, G, Z4, Y4, 4, "silu", *b4)


def test_without_saved_z():
    X, A, B, _ = inputs(200, 256, 512)
    O, Z, Y = tp.gated_forward(X, A, B, 2)
    O2, none, Y2 = tp.gated_forward(X, A, B, 2, save=False)
    assert none is None and torch.equal(O, O2) and torch.equal(Y, Y2)


def test_gradients_are_added():
    X, A, B, G = inputs(200, 136, 272, seed=3)
    _, Z, Y = tp.gated_forward(X, A, B, 2)
    dA, dB = (torch.randn(*v.shape, device="cuda") for v in (A, B))
    old = host(dA), host(dB)
    got = tp.gated_backward(X, A, B, G, Z, Y, 2, wgrad="f32_add", dA=dA, dB=dB)
    assert got[1] is dA and got[2] is dB
    check_backward(X, A, B, G, Z, Y, 2, "silu", *got, before=old)


def test_large_gates():
    # exp(-g) past fp32 on one side and nothing on the other: silu is 0 or g, its slope 0 or 1
    X, A, B, G = inputs(64, 64, 128)
    A[:, :128] *= 200
    O, Z, Y = tp.gated_forward(X, A, B, 1)
    assert host(Z[:, :128]).min() < -300 and host(Z[:, :128]).max() > 300
    check_forward(X, A, B, 1, "silu", O, Z, Y)
    check_backward(X, A, B, G, Z, Y, 1, "silu", *tp.gated_backward(X, A, B, G, Z, Y, 1))


def test_what_a_row_holds_stays_in_it():
    # a row of infinities and NaN changes no other row, forward and in dX
    X, A, B, G = inputs(140, 128, 256)
    want = tp.gated_forward(X, A, B, 2)
    gwant = tp.gated_backward(X, A, B, G, want[1], want[2], 2)
    X2, G2 = X.clone(), G.clone()
    X2[77], G2[77] = float("nan"), float("inf")
    got = tp.gated_forward(X2, A, B, 2)
    keep = torch.arange(140, device="cuda") != 77
    for a, b in zip(want, got):
        assert torch.equal(a[keep], b[keep]) and torch.isnan(b[77]).all()
    gx = tp.gated_backward(X, A, B, G2, want[1], want[2], 2)[0]
    assert torch.equal(gx[keep], gwant[0][keep]) and not torch.isfinite(gx[77]).any()


def test_neighbouring_shards_do_not_leak():
    # shards of 40 columns end inside every column block: what is past a shard's end is its neighbour's
    X, A, B, _ = inputs(30, 64, 120)
    want = tp.gated_forward(X, A, B, 3)
    A2 = A.clone()
    A2[:, 80:160] = float("nan")                                   # all of shard 1
    got = tp.gated_forward(X, A2, B, 3)
    for a, b, w in ((want[2], got[2], 40), (want[1], got[1], 80)):
        assert torch.equal(a[:, :w], b[:, :w]) and torch.equal(a[:, 2 * w:], b[:, 2 * w:])
        assert torch.isnan(b[:, w:2 * w]).all()


def test_no_tokens():
    X, A, B, G = inputs(0, 64, 128)
    O, Z, Y = tp.gated_forward(X, A, B, 2)
    assert O.shape == (0, 64) and Z.shape == (0, 256) and Y.shape == (0, 128)
    for wgrad in ("f32", "operand"):
        dX, dA, dB = tp.gated_backward(X, A, B, G, Z, Y, 2, wgrad=wgrad)
        assert dX.shape == (0, 64) and not dA.any() and not dB.any()
    dA, dB = torch.ones(64, 256, device="cuda"), torch.ones(128, 64, device="cuda")
    tp.gated_backward(X, A, B, G, Z, Y, 2, wgrad="f32_add", dA=dA, dB=dB)
    assert (dA == 1).all() and (dB == 1).all()


@pytest.mark.parametrize("n", [4, 300])
def test_on_another_stream_and_from_a_graph(n):
    X, A, B, G = inputs(n, 256, 512)
    want = tp.gated_forward(X, A, B, 2)
    gwant = tp.gated_backward(X, A, B, G, want[1], want[2], 2)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = tp.gated_forward(X, A, B, 2, stream=side)
    ggot = tp.gated_backward(X, A, B, G, got[1], got[2], 2, stream=side)
    side.synchronize()
    for a, b in zip(want + gwant, got + ggot):
        assert torch.equal(a, b)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cap = tp.gated_forward(X, A, B, 2)
        gcap = tp.gated_backward(X, A, B, G, cap[1], cap[2], 2)
    for _ in range(2):
        X.copy_(X.flip(0))
        G.copy_(G.flip(0))
        graph.replay()
    torch.cuda.synchronize()
    for a, b in zip(want + gwant, cap + gcap):
        assert torch.equal(a, b)
    tp.tpmlp_device_status()


@pytest.mark.parametrize("n", [8, 200])
def test_two_calls_at_once(n):
    # calls on two streams keep to their own workspaces
    ins = [inputs(n, 512, 1024, seed) for seed in (1, 2)]
    want = [tp.gated_forward(*i[:3], 2) for i in ins]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in ins]
    for _ in range(5):
        got = [tp.gated_forward(*i[:3], 2, stream=s) for i, s in zip(ins, streams)]
        torch.cuda.synchronize()
        for w, g in zip(want, got):
            assert all(torch.equal(a, b) for a, b in zip(w, g))


# ----------------------------------------------------------------------- sums split across the SMs

# Few tokens or small outputs with a long sum (n, d, m, t), all on single SMs. FC1 split, with shards of whole column blocks and with
# ragged ones; unsplit; on the SM-pair GEMM. FC2 and dX split; of two and three tiles of tokens; output columns that end inside a
# tile and inside its first half.
SPLIT = [(5, 4096, 256, 2), (5, 4096, 264, 3), (150, 4096, 1000, 5), (200, 16384, 1024, 1), (4, 512, 16384, 8),
         (33, 264, 8192, 4), (300, 256, 4096, 2), (520, 512, 4096, 1), (600, 264, 4096, 1), (130, 1024, 8192, 1),
         (1, 72, 8192, 1)]


@pytest.mark.parametrize("shape", SPLIT)
def test_split_sums(shape):
    run_and_check(*shape, kind=ACTS[shape[0] % 3], wgrad="operand", seed=shape[0])


@pytest.mark.parametrize("shape", [(5, 4096, 256, 2), (200, 4096, 768, 4), (300, 256, 4096, 2)])
def test_split_sums_are_the_same_every_time(shape):
    n, d, m, t = shape
    X, A, B, G = inputs(n, d, m)
    want = tp.gated_forward(X, A, B, t)
    gwant = tp.gated_backward(X, A, B, G, want[1], want[2], t)
    for _ in range(10):
        got = tp.gated_forward(X, A, B, t)
        ggot = tp.gated_backward(X, A, B, G, want[1], want[2], t)
        assert all(torch.equal(a, b) for a, b in zip(want + gwant, got + ggot))


def on_gpu(X, A, B, kind):
    """Y and O in 64 bits, and the deviations that check_forward allows (t = 1), for sizes that are too large for the host."""
    x, a, b = (v.double() for v in (X, A, B))
    m = b.shape[0]
    z, slip = x @ a, acc(a.shape[0]) * (x.abs() @ a.abs())
    g, u = z[:, :m], z[:, m:]
    assert kind == "silu"
    sig = torch.sigmoid(g)
    y = g * sig * u
    off = 1.2 * slip[:, :m] * u.abs() + (g * sig).abs() * slip[:, m:] + 2.0 ** -20 * (1 + g.abs()) * u.abs()
    o = y @ b
    dev = ((U / 3 ** 0.5 * y) ** 2 + off ** 2) @ (b * b)
    return y, U * y.abs() + 2 * off, o, U * o.abs() + 7 * dev.sqrt() + acc(m) * (y.abs() @ b.abs())


@pytest.mark.parametrize("shape", [(3, 32768, 1024), (200, 16384, 16384), (64, 4096, 16384)])
def test_unsplit_sums_of_large_weights(shape):
    # many column tiles: the products' own epilogues write O and Y, on single SMs and on pairs
    n, d, m = shape
    X, A, B, _ = inputs(n, d, m)
    O, Z, Y = tp.gated_forward(X, A, B, 1, "silu", save=False)
    y, y_bound, o, o_bound = on_gpu(X, A, B, "silu")
    assert ((Y.double() - y).abs() <= y_bound).all() and ((O.double() - o).abs() <= o_bound).all()
    O2, Z2, Y2 = tp.gated_forward(X, A, B, 1, "silu")
    assert torch.equal(O, O2) and torch.equal(Y, Y2)
    z = X.double() @ A.double()
    assert ((Z2.double() - z).abs() <= U * z.abs() + acc(d) * (X.double().abs() @ A.double().abs())).all()


@pytest.mark.parametrize("shape", [(8, 20000, 1024), (1000, 5000, 8192), (200, 1024, 16384)])
def test_products_of_many_columns_and_of_several_rounds(shape):
    # FC2 and dX unsplit, split over three rounds of CTAs, and split with hundreds of k-blocks each
    n, d, m = shape
    X, A, B, G = inputs(n, d, m)
    O, Z, Y = tp.gated_forward(X, A, B, 1, "silu")
    y, y_bound, o, o_bound = on_gpu(X, A, B, "silu")
    assert ((Y.double() - y).abs() <= y_bound).all() and ((O.double() - o).abs() <= o_bound).all()
    dX = tp.gated_backward(X, A, B, G, Z, Y, 1, wgrad="operand")[0]
    tp.tpmlp_device_status()
    zz = Z.double().requires_grad_()
    D, = torch.autograd.grad(torch.nn.functional.silu(zz[:, :m]) * zz[:, m:], zz, G.double() @ B.double().T)
    a = A.double()
    want = D @ a.T
    # D is rounded once, and its dY is a sum of d terms: as one more rounding of the magnitudes that it is made of
    mag = torch.cat([zz[:, m:].abs(), zz[:, :m].abs() + 1], 1) * (G.double().abs() @ B.double().abs().T).repeat(1, 2)
    dev = ((U / 3 ** 0.5 * D) ** 2 + (1.2 * acc(d) * mag) ** 2) @ (a * a).T
    assert ((dX.double() - want).abs() <= U * want.abs() + 7 * dev.sqrt() + acc(2 * m) * (D.abs() @ a.abs().T)).all()
