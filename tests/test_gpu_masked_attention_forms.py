"""Masked attention in the forms that have a kernel, or an issue loop, of their own: every mask and arbitrary intervals with
heads of 64 and of 128 columns, with and without a cap and a bias, forward and backward, against the float64 oracle."""
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

import tensor_transformer_mlp_gb300 as tp
from oracle import masked_attention as oma
from test_gpu_masked_attention import SLACK, U, _check, _draw, _gpu_ranges, _hold, _masks, _np

pytestmark = pytest.mark.gpu
FORMS = [(64, 0.0, False), (64, 20.0, True), (128, 0.0, False), (128, 20.0, False), (128, 0.0, True), (128, 20.0, True)]
SLOPES = [0.05, 0.01]


@pytest.mark.parametrize("name", list(_masks(2, 64)))
@pytest.mark.parametrize("hd,cap,bias", FORMS)
def test_every_mask_in_every_kernel(hd, cap, bias, name):
    s = 385
    mask = _masks(2, s, seed=hd)[name]
    q, k, v, dO = _draw(hd, 2, s, 2, 1, hd)
    ranges = oma.key_ranges(2, s, **mask)
    assert np.array_equal(_gpu_ranges(2, s, mask).cpu().numpy(), ranges)
    _check(q, k, v, dO, ranges, cap=cap, slopes=SLOPES if bias else None)


@pytest.mark.parametrize("seed", [0, 1])
@pytest.mark.parametrize("hd,cap,bias", FORMS)
def test_arbitrary_intervals(hd, cap, bias, seed):
    # no order between neighbours, empty rows among them, ends outside the sequence
    s = 333
    r = np.random.default_rng(seed + hd)
    ranges = np.sort(r.integers(-40, s + 40, (2, s, 2)), axis=2).astype(np.int32)
    ranges[:, r.integers(0, s, 60)] = 0
    ranges[0, 130:262] = [7, 7]
    ranges[1, 5] = [200, 100]
    ranges[1, 6] = [-2 ** 31, 2 ** 31 - 1]
    q, k, v, dO = _draw(seed, 2, s, 2, 1, hd)
    _check(q, k, v, dO, ranges, cap=cap, slopes=SLOPES if bias else None)


@pytest.mark.parametrize("hd,cap,bias", FORMS)
def test_key_tiles_that_neither_query_tile_sees(hd, cap, bias):
    # the two tiles of a piece far apart, either way round, next to pieces with one tile, and with none
    s = 1290
    ranges = np.zeros((1, s, 2), np.int32)
    ranges[0, :128] = [3, 60]
    ranges[0, 128:256] = [900, 1000]
    ranges[0, 256:384] = [1100, s]
    ranges[0, 384:512] = [130, 131]
    ranges[0, 520:530] = [0, s]
    ranges[0, 768:800] = [640, 700]
    ranges[0, 1024:1152:3] = [5, 1200]
    q, k, v, dO = _draw(hd + 5, 1, s, 2, 2, hd, "packed")
    _check(q, k, v, dO, ranges, cap=cap, slopes=SLOPES if bias else None)


@pytest.mark.parametrize("hd", [64, 128])
def test_offsets_past_32_bits_in_every_output(hd):
    # token rows of 128 KB: the last rows of every tensor lie 5 GB behind the first
    s, ld = 40000, 65536
    big = torch.empty(s, ld, dtype=torch.bfloat16, device="cuda")
    gen = torch.Generator("cuda").manual_seed(3)
    big[:, :4 * hd] = torch.randn(s, 4 * hd, generator=gen, device="cuda").bfloat16()
    q, k, v, dO = (big[:, n * hd:(n + 1) * hd].view(1, s, 1, hd) for n in range(4))
    o, dq, dk, dv = (big[:, ld - n * hd:ld - (n - 1) * hd or None].view(1, s, 1, hd) for n in range(1, 5))
    ranges = tp.attention_key_ranges(1, s, window=50, device="cuda")
    _, lse = tp.masked_attention_forward(q, k, v, ranges, o=o)
    tp.masked_attention_backward(q, k, v, ranges, o, lse, dO, dq=dq, dk=dk, dv=dv)
    torch.cuda.synchronize()
    tp.tpmlp_device_status()
    for rows in (slice(0, 300), slice(s // 2, s // 2 + 300), slice(s - 300, s)):   # alone, as a sequence of their own
        sub = [_np(t[:, rows].clone()) for t in (q, k, v, dO)]
        f = oma.attention(*sub[:3], oma.key_ranges(1, 300, window=50), hd ** -0.5, dO=sub[3])
        far = slice(0 if rows.start == 0 else 50, 300 if rows.stop == s else 250)   # whose keys, or queries, are all there
        tol = {"o": U * (f["o_abs"] + np.abs(f["o"])) + SLACK * f["o_abs"],
               "dv": U * (f["dv_abs"] + np.abs(f["dv"])) + SLACK * f["dv_abs"]}
        for name in ("dq", "dk"):
            tol[name] = U * (f[name + "_d"] + f[name + "_abs"] + np.abs(f[name])) + SLACK * f[name + "_p"]
        for name, got in (("o", o), ("dq", dq), ("dk", dk), ("dv", dv)):
            _hold(name, got[:, rows][:, far], f[name][:, far], tol[name][:, far])


COLD = """
import torch, tensor_transformer_mlp_gb300 as tp
q, k, v, do = (torch.randn(1, 300, 2, {hd}, device="cuda").bfloat16() for _ in range(4))
g = torch.ones({hd}, device="cuda")
cos, sin = tp.rope_tables(300, {hd}, device="cuda")
ids = torch.zeros(1, 300, dtype=torch.int32, device="cuda")

def step():
    r = tp.attention_key_ranges(1, 300, doc_ids=ids)
    qn, kn = tp.qk_norm_rope(q, k, g, g, cos, sin)
    o, lse = tp.masked_attention_forward(qn, kn, v, r)
    dq, dk, dv = tp.masked_attention_backward(qn, kn, v, r, o, lse, do)
    return (o, lse, dv) + tp.qk_norm_rope_backward(q, k, g, g, cos, sin, dq, dk)

torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    held = step()
graph.replay()
torch.cuda.synchronize()
for a, b in zip(held, step()):
    assert torch.equal(a, b)
tp.tpmlp_device_status()
print("same")
"""


@pytest.mark.parametrize("hd", [64, 128])
def test_a_process_whose_first_calls_are_captured(hd):
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    out = subprocess.run([sys.executable, "-c", COLD.format(hd=hd)], cwd=root, capture_output=True, text=True, timeout=300)
    assert out.returncode == 0 and out.stdout.strip() == "same", out.stderr[-2000:]
