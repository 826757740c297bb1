"""Float64 oracle of the per-head norm of queries and keys with the position rotation (test infrastructure only).

Method: RMSNorm (the "RMSNorm" section of the "Megatron 训练" notes, as in ``oracle.rmsnorm``) over the columns of one
head, then a rotation of the first rot columns in pairs. With u = x r gamma, r = 1 / sqrt(mean(x^2) + eps), the pair
(a, b) with angle t becomes (a cos t - b sin t, b cos t + a sin t); pairs are columns (i, i + rot/2) in the half style
and (2i, 2i + 1) in the interleaved one. The angles' cosines and sines come from tables, row = position.

The rotation is written here as a matrix per position, so that its transpose is the backward's.
"""
from __future__ import annotations

import numpy as np


def rotation_matrix(cos_row, sin_row, hd: int, style: str) -> np.ndarray:
    """R [hd, hd] with y = R u for one position."""
    half = len(cos_row)
    R = np.eye(hd)
    for i in range(half):
        a, b = (i, i + half) if style == "half" else (2 * i, 2 * i + 1)
        c, s = float(cos_row[i]), float(sin_row[i])
        R[a, a], R[a, b], R[b, a], R[b, b] = c, -s, s, c
    return R


def _matrices(cos, sin, pos, hd, style):
    """[tokens, hd, hd]; zero for a negative position."""
    known = {}
    out = np.zeros((len(pos), hd, hd))
    for t, p in enumerate(pos):
        if p >= 0:
            if p not in known:
                known[p] = rotation_matrix(cos[p], sin[p], hd, style)
            out[t] = known[p]
    return out


def forward(x, gamma, eps: float, cos, sin, pos, style: str) -> np.ndarray:
    """x [tokens, heads, hd] -> y; tokens of negative position give zeros."""
    x = np.asarray(x, np.float64)
    r = 1.0 / np.sqrt((x * x).mean(axis=-1, keepdims=True) + eps)
    u = x * r * np.asarray(gamma, np.float64)
    return np.einsum("tij,thj->thi", _matrices(cos, sin, pos, x.shape[-1], style), u)


def backward(x, gamma, eps: float, cos, sin, pos, style: str, dy):
    """Returns dx and dgamma (summed over tokens and heads)."""
    x, dy = np.asarray(x, np.float64), np.asarray(dy, np.float64)
    live = (np.asarray(pos) >= 0)[:, None, None]
    du = np.einsum("tji,thj->thi", _matrices(cos, sin, pos, x.shape[-1], style), dy)
    r = 1.0 / np.sqrt((x * x).mean(axis=-1, keepdims=True) + eps)
    xhat = x * r
    g = du * np.asarray(gamma, np.float64)
    dx = r * (g - xhat * (g * xhat).mean(axis=-1, keepdims=True)) * live
    return dx, (du * xhat * live).sum(axis=(0, 1))
