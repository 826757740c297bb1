"""The gated block's FC1 of few tokens without a split, on single SMs and on pairs, with shards that end inside a block of columns.
Each test names the form that its sizes run on and looks it up in the plan. Tolerances as in test_gpu_gated.py, in 64 bits on the
GPU, because the sizes are too large for the host."""
import pytest
import torch

import few_rows_plan
import tensor_transformer_mlp_gb300 as tp

pytestmark = pytest.mark.gpu

U = 2.0 ** -8
TANH = 2.0 ** -10.9
ACTS = ["silu", "gelu_tanh", "gelu_erf"]


def acc(k):
    return (k / 16 + 1) * 2.0 ** -22


def inputs(n, d, m, seed):
    gen = torch.Generator("cuda").manual_seed(seed)

    def draw(scale, *shape):
        return (scale * torch.randn(*shape, generator=gen, device="cuda")).bfloat16()
    return draw(1, n, d), draw(d ** -0.5, d, 2 * m), draw(m ** -0.5, m, d)


def act64(g, kind):
    """act(g) and what the kernel's act may be off by."""
    if kind == "silu":
        return g * torch.sigmoid(g), 2.0 ** -20 * (1 + g.abs())
    if kind == "gelu_erf":
        return 0.5 * g * (1 + torch.erf(g * 0.5 ** 0.5)), 2.0 ** -20 * (1 + g.abs())
    th = torch.tanh((2 / torch.pi) ** 0.5 * (g + 0.044715 * g ** 3))
    return 0.5 * g * (1 + th), 0.5 * (g * th).abs() * TANH + 2.0 ** -20 * (1 + g.abs())


def parts(z, t):
    """The gate and up columns of the shards of Z."""
    v = z.unflatten(1, (t, 2, -1))
    return v[:, :, 0].flatten(1), v[:, :, 1].flatten(1)


def run_and_check(n, d, m, t):
    X, A, B = inputs(n, d, m, seed=n + d + t)
    x, a, b = (v.double() for v in (X, A, B))
    z, slip = x @ a, acc(d) * (x.abs() @ a.abs())
    (g, u), (slip_g, slip_u) = parts(z, t), parts(slip, t)
    for kind in ACTS:
        O, Z, Y = tp.gated_forward(X, A, B, t, kind)
        tp.tpmlp_device_status()
        assert ((Z.double() - z).abs() <= U * z.abs() + slip).all(), kind
        f, f_off = act64(g, kind)
        y, off = f * u, 1.2 * slip_g * u.abs() + f.abs() * slip_u + f_off * u.abs()      # |act'| < 1.2
        assert ((Y.double() - y).abs() <= U * y.abs() + 2 * off).all(), kind
        o, dev = y @ b, ((U / 3 ** 0.5 * y) ** 2 + off ** 2) @ (b * b)
        assert ((O.double() - o).abs() <= U * o.abs() + 7 * dev.sqrt() + acc(m) * (y.abs() @ b.abs())).all(), kind
        O2, none, Y2 = tp.gated_forward(X, A, B, t, kind, save=False)
        assert none is None and torch.equal(O, O2) and torch.equal(Y, Y2), kind


# (n, d, m, t). Shards that end inside a block of 64 columns: 8 of 1376, 3 of 3640, 8 of 1368, 4 of 2736. Whole ones whose last tile
# has 64 of 256 columns, and 7 of 2048. Rows of A that end inside a k-block. Tokens on both sides of steps of 16 and 32.
PAIRS = [(130, 8192, 11008, 8), (144, 8192, 11008, 1), (150, 4096, 11008, 8), (161, 4096, 11008, 1), (170, 4096, 10920, 3),
         (200, 4096, 10944, 8), (200, 4104, 11072, 1), (225, 4104, 14336, 7), (240, 8192, 10944, 4)]


@pytest.mark.parametrize("shape", PAIRS)
def test_pairs_of_sms(shape):
    plan, = few_rows_plan.fc1([shape])
    assert plan["takes"] and plan["ranks"] == 2 and plan["splits"] == 1 and plan["nt"] % 32 == 0
    run_and_check(*shape)


SINGLES = [(1, 4096, 11072, 1), (4, 1032, 10944, 4), (64, 4096, 10960, 2), (97, 4096, 10944, 8), (130, 2056, 10944, 4)]


@pytest.mark.parametrize("shape", SINGLES)
def test_single_sms(shape):
    plan, = few_rows_plan.fc1([shape])
    assert plan["takes"] and plan["ranks"] == 1 and plan["splits"] == 1
    run_and_check(*shape)


@pytest.mark.parametrize("shape", [(4, 8192, 8448, 32), (128, 4096, 8448, 32)])
def test_many_ragged_shards(shape):
    plan, = few_rows_plan.fc1([shape])
    assert plan["takes"] and plan["splits"] == 1 and plan["unit"] == 264
    run_and_check(*shape)
