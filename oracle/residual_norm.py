"""Float64 oracle of the norms before and after a block: r = alpha x + gate * rmsnorm(y) gamma_post, u = rmsnorm(r) gamma_pre,
and its gradients. x, y [b, s, h]; gate [b, h] or None; a missing gain is None (no norm at that place). Test infrastructure only.
"""
import numpy as np


def _root(v, eps):
    return 1.0 / np.sqrt((v * v).mean(-1, keepdims=True) + eps)


def _f64(*vs):
    return tuple(None if v is None else np.asarray(v, np.float64) for v in vs)


def forward(x, y, post, gate, pre, alpha, eps):
    """(r, u); u None without pre."""
    x, y, post, gate, pre = _f64(x, y, post, gate, pre)
    p = y if post is None else y * _root(y, eps) * post
    r = alpha * x + (p if gate is None else gate[:, None] * p)
    return r, None if pre is None else r * _root(r, eps) * pre


def _norm_backward(v, gamma, dout, eps):
    root = _root(v, eps)
    hat, g = v * root, dout * gamma
    return root * (g - hat * (g * hat).mean(-1, keepdims=True)), (dout * hat).sum((0, 1))


def backward(y, r, dr, du, post, gate, pre, alpha, eps):
    """{dx, dy, dpost, dgate, dpre}, without those of missing gains and gate."""
    y, r, dr, du, post, gate, pre = _f64(y, r, dr, du, post, gate, pre)
    out = {}
    g = np.zeros_like(du) if dr is None else dr
    if pre is not None:
        more, out["dpre"] = _norm_backward(r, pre, du, eps)
        g = g + more
    out["dx"] = alpha * g
    if gate is not None:
        p = y if post is None else y * _root(y, eps) * post
        out["dgate"] = (g * p).sum(1)
        g = gate[:, None] * g
    out["dy"] = g
    if post is not None:
        out["dy"], out["dpost"] = _norm_backward(y, post, g, eps)
    return out
