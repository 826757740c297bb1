"""Float64 oracle of masked attention and of the key ranges of its masks (test infrastructure only).

Per sequence and query head, with the keys j of the query's range [lo_i, hi_i):

    y_ij = c(scale q_i.k_j) - slope |i - j|,   c(x) = cap tanh(x / cap) (x when cap is 0)
    lse_i = log sum_j exp(y_ij),   P_ij = exp(y_ij - lse_i),   o_i = sum_j P_ij v_j

(a query without keys: o = 0, lse = -inf), and from dO the gradients of o written out as the chain rule gives them:

    dV_j = sum_i P_ij dO_i,   dY_ij = P_ij (dO_i.v_j - sum_j' P_ij' dO_i.v_j'),   dX_ij = scale c' dY_ij,
    dQ_i = sum_j dX_ij k_j,   dK_j = sum_i dX_ij q_i,

a key or value head collecting its query heads (softmax and its gradient as in the "Attention 层" section of the
"Megatron 训练" notes, which has no mask). Beside each result stands the sum of its terms' magnitudes, from which
tests derive how far roundings can move it.
"""
from __future__ import annotations

import numpy as np


def key_ranges(b: int, s: int, doc_ids=None, prefix_len=None, causal: bool = True, window: int = 0) -> np.ndarray:
    """[b, s, 2] key intervals, pair by pair from the mask's definition."""
    out = np.zeros((b, s, 2), np.int32)
    for bi in range(b):
        ids = np.zeros(s, np.int64) if doc_ids is None else np.asarray(doc_ids)[bi]
        doc = np.concatenate([[0], np.cumsum(ids[1:] != ids[:-1])]) if s else ids
        prefix = 0 if prefix_len is None else int(prefix_len[bi])
        j = np.arange(s)
        for i in range(s):
            seen = (doc == doc[i]) & (ids[i] >= 0)
            if causal:
                seen &= (j <= i) | (j < prefix)
            if window:
                seen &= i - j < window
                if not causal:
                    seen &= j - i < window
            at = np.flatnonzero(seen)
            if len(at):
                assert at[-1] - at[0] + 1 == len(at)
                out[bi, i] = at[0], at[-1] + 1
    return out


def attention(q, k, v, ranges, scale: float, cap: float = 0.0, slopes=None, dO=None) -> dict[str, np.ndarray]:
    """q [b, s, heads, hd], k, v [b, s, kv, hd]. Returns o, lse and, with dO, dq, dk, dv; the magnitudes of their
    terms: o_abs = sum P|v|, dv_abs, and dq_move, dk_move: the sums of |k| (|q|) times
    scale c' P (sum |dO| (o_abs + |o|), sum |dO||v|)."""
    q, k, v = (np.asarray(a, np.float64) for a in (q, k, v))
    b, s, heads, hd = q.shape
    kv = k.shape[2]
    group = heads // kv
    f = {"o": np.zeros(q.shape), "lse": np.full((b, heads, s), -np.inf), "o_abs": np.zeros(q.shape),
         "y_abs": np.zeros((b, heads, s))}
    if dO is not None:
        dO = np.asarray(dO, np.float64)
        for n in ("dq", "dq_d", "dq_p", "dq_abs"):
            f[n] = np.zeros(q.shape)
        for n in ("dk", "dk_d", "dk_p", "dk_abs", "dv", "dv_abs"):
            f[n] = np.zeros(k.shape)
    j = np.arange(s)
    for bi in range(b):
        r = np.asarray(ranges)[bi]
        seen = (j >= r[:, :1]) & (j < r[:, 1:])
        for h in range(heads):
            g = h // group
            x = scale * q[bi, :, h] @ k[bi, :, g].T
            mag = scale * np.abs(q[bi, :, h]) @ np.abs(k[bi, :, g]).T
            dc = np.ones_like(x)
            if cap:
                t = np.tanh(x / cap)
                x, dc = cap * t, 1 - t * t
            if slopes is not None:
                x = x - float(slopes[h]) * np.abs(j[:, None] - j)
            x = np.where(seen, x, -np.inf)
            top = x.max(axis=1, initial=-np.inf)
            safe = np.where(np.isfinite(top), top, 0.0)
            e = np.exp(x - safe[:, None])
            total = e.sum(axis=1)
            with np.errstate(divide="ignore"):
                f["lse"][bi, h] = np.where(total > 0, safe + np.log(total), -np.inf)
            P = e / np.where(total > 0, total, 1.0)[:, None]
            f["y_abs"][bi, h] = np.where(seen, mag, 0.0).max(axis=1, initial=0.0)
            f["o"][bi, :, h] = P @ v[bi, :, g]
            f["o_abs"][bi, :, h] = P @ np.abs(v[bi, :, g])
            if dO is None:
                continue
            G = dO[bi, :, h]
            dP = G @ v[bi, :, g].T
            dY = P * (dP - (P * dP).sum(axis=1, keepdims=True))
            dX = scale * dc * dY
            f["dq"][bi, :, h] = dX @ k[bi, :, g]
            f["dk"][bi, :, g] += dX.T @ q[bi, :, h]
            f["dv"][bi, :, g] += P.T @ G
            f["dv_abs"][bi, :, g] += P.T @ np.abs(G)
            # |dX| enters once more for the rounding of dX; D moves with o's roundings; dP and D themselves
            # are fp32 sums
            d_move = (np.abs(G) * (f["o_abs"][bi, :, h] + 2 * np.abs(f["o"][bi, :, h]))).sum(axis=1, keepdims=True)
            W = scale * dc * P
            p_mag = W * (np.abs(G) @ np.abs(v[bi, :, g]).T + (np.abs(G) * f["o_abs"][bi, :, h]).sum(axis=1, keepdims=True))
            ak, aq = np.abs(k[bi, :, g]), np.abs(q[bi, :, h])
            f["dq_d"][bi, :, h] = (W * d_move) @ ak
            f["dq_p"][bi, :, h] = p_mag @ ak
            f["dq_abs"][bi, :, h] = np.abs(dX) @ ak
            f["dk_d"][bi, :, g] += (W * d_move).T @ aq
            f["dk_p"][bi, :, g] += p_mag.T @ aq
            f["dk_abs"][bi, :, g] += np.abs(dX).T @ aq
    return f
