"""Float64 oracle of the gated feed-forward block: Z = X A, Y = act(Z_gate) * Z_up, O = Y B and its gradients.

Shard i of t holds m/t gate columns, then m/t up columns, from column 2 i m/t of A and Z on. Test infrastructure only:
nothing outside tests and smoke() imports it.
"""
import numpy as np

from . import mlp


def act(z, kind):
    if kind == "silu":
        return z / (1.0 + np.exp(-z))
    return mlp.gelu(z, kind.removeprefix("gelu_"))


def act_grad(z, kind):
    if kind == "silu":
        s = 1.0 / (1.0 + np.exp(-z))
        return s * (1.0 + z * (1.0 - s))
    return mlp.gelu_grad(z, kind.removeprefix("gelu_"))


def columns(m, t):
    """The gate and up columns of Z (or A) of the m columns of Y."""
    y = np.arange(m)
    shard, j = y // (m // t), y % (m // t)
    gate = shard * 2 * (m // t) + j
    return gate, gate + m // t


def forward(X, A, B, t, kind):
    """{Z, Y, O} in float64."""
    X, A, B = (np.asarray(v, np.float64) for v in (X, A, B))
    gate, up = columns(B.shape[0], t)
    Z = X @ A
    Y = act(Z[:, gate], kind) * Z[:, up]
    return {"Z": Z, "Y": Y, "O": Y @ B}


def backward(X, A, B, G, Z, Y, t, kind):
    """{dX, dA, dB, D} from the saved Z and Y."""
    X, A, B, G, Z, Y = (np.asarray(v, np.float64) for v in (X, A, B, G, Z, Y))
    gate, up = columns(B.shape[0], t)
    dY = G @ B.T
    D = np.empty_like(Z)
    D[:, gate] = dY * Z[:, up] * act_grad(Z[:, gate], kind)
    D[:, up] = dY * act(Z[:, gate], kind)
    return {"D": D, "dX": D @ A.T, "dA": X.T @ D, "dB": Y.T @ G}
