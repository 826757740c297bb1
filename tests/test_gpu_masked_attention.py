"""GPU parity of masked attention, its gradients and the key ranges of its masks against the float64 oracle.

Tolerances, element by element, from what is rounded (u = 2^-8, half a bf16 step; P and dX go to the tensor core in
bf16, o and the gradients are stored in bf16, everything else is fp32):
  o:   u (sum P|v| + |o|)
  lse: the score's fp32 sum, hd 2^-24 sum|q||k| scale, plus 2^-20 for exponent, logarithm and the row's sum
  dv:  u (sum P|dO| + |dv|)
  dX:  D = dO.o moves with o's roundings, u sum|dO| (sum P|v| + 2|o|) in all, and dX itself is rounded once:
       dq: u (sum W|k| d_move + sum |dX||k| + |dq|), W = scale c' P; dk likewise over the queries
An fp32 slack of 2^-12 of the terms' magnitudes stands for the recomputed P (its exponent is off by the errors of
the score and of lse, up to about 1e-4 here) and for fp32 sums; it is 1/16 of u.
"""
import math

import numpy as np
import pytest
import torch

import tensor_transformer_mlp_gb300 as tp
from oracle import masked_attention as oma
from oracle import qk_norm_rope as oqr

pytestmark = pytest.mark.gpu

U = 2.0 ** -8
SLACK = 2.0 ** -12


def _draw(seed, b, s, heads, kv, hd, layout="separate", std=1.0):
    """q, k, v views on the GPU and dO."""
    gen = torch.Generator("cuda").manual_seed(seed)
    rand = lambda *shape: (std * torch.randn(*shape, generator=gen, device="cuda")).bfloat16()  # noqa: E731
    if layout == "packed":       # the attention block's QKV matrix: [q | k | v] per head
        assert heads == kv
        m = rand(b, s, heads, 3, hd)
        q, k, v = m[:, :, :, 0], m[:, :, :, 1], m[:, :, :, 2]
    elif layout == "joined":     # all queries, then all keys, then all values
        m = rand(b, s, (heads + 2 * kv) * hd)
        q, k, v = m.split([heads * hd, kv * hd, kv * hd], -1)
        q, k, v = q.unflatten(-1, (heads, hd)), k.unflatten(-1, (kv, hd)), v.unflatten(-1, (kv, hd))
    else:
        q, k, v = rand(b, s, heads, hd), rand(b, s, kv, hd), rand(b, s, kv, hd)
    return q, k, v, rand(b, s, heads, hd)


def _np(t):
    return t.double().cpu().numpy()


def _hold(name, got, ref, tol):
    got = _np(got)
    assert np.isfinite(got).all(), f"{name}: not finite"
    over = np.abs(got - ref) - tol
    at = np.unravel_index(np.argmax(over), over.shape)
    assert over[at] <= 0, f"{name}{list(map(int, at))}: {got[at]} for {ref[at]}, tolerance {tol[at]}"


def _check(q, k, v, dO, ranges, cap=0.0, slopes=None, scale=None, backward=True):
    hd = q.shape[-1]
    sc = 1 / math.sqrt(hd) if scale is None else scale
    rng = torch.from_numpy(np.ascontiguousarray(ranges)).cuda()
    sl = None if slopes is None else torch.tensor(slopes, dtype=torch.float32, device="cuda")
    o, lse = tp.masked_attention_forward(q, k, v, rng, scale=scale, softcap=cap, slopes=sl)
    grads = tp.masked_attention_backward(q, k, v, rng, o, lse, dO, scale=scale, softcap=cap, slopes=sl) if backward else ()
    torch.cuda.synchronize()
    tp.tpmlp_device_status()
    f = oma.attention(_np(q), _np(k), _np(v), ranges, sc, cap, slopes, _np(dO) if backward else None)
    tiny = 1e-30
    _hold("o", o, f["o"], U * (f["o_abs"] + np.abs(f["o"])) + SLACK * f["o_abs"] + tiny)
    got, none = lse.double().cpu().numpy(), np.isneginf(f["lse"])
    assert np.array_equal(np.isneginf(got), none)
    tol = hd * 2.0 ** -24 * f["y_abs"] + 2.0 ** -20 * (1 + np.abs(np.where(none, 0, f["lse"]))) + 2.0 ** -21 * cap
    if slopes is not None:  # a row's part and a column's part, up to 256 slope in the tiles near a row; three roundings
        tol = tol + 3 * 2.0 ** -24 * 256 * np.abs(slopes).max()
    assert (np.abs(np.where(none, 0, got) - np.where(none, 0, f["lse"])) <= tol).all()
    if not backward:
        return o, lse
    dq, dk, dv = grads
    _hold("dv", dv, f["dv"], U * (f["dv_abs"] + np.abs(f["dv"])) + SLACK * f["dv_abs"] + tiny)
    for name, g in (("dq", dq), ("dk", dk)):
        _hold(name, g, f[name], U * (f[name + "_d"] + f[name + "_abs"] + np.abs(f[name])) + SLACK * f[name + "_p"] + tiny)
    return o, lse, dq, dk, dv


def _docs(b, s, n, seed, pad=True):
    r = np.random.default_rng(seed)
    ids = np.full((b, s), -1, np.int32)
    for bi in range(b):
        end = s - int(r.integers(0, s // 4 + 1)) if pad else s
        cuts = np.sort(r.integers(0, end + 1, n - 1))
        for d, (lo, hi) in enumerate(zip([0, *cuts], [*cuts, end])):
            ids[bi, lo:hi] = d * 3
    return ids


def _masks(b, s, seed=0):
    """name -> arguments of the key ranges."""
    r = np.random.default_rng(seed)
    return {
        "full": dict(causal=False),
        "causal": dict(),
        "window": dict(window=max(1, s // 3)),
        "window-of-one": dict(window=1),
        "both-sides": dict(causal=False, window=max(2, s // 5)),
        "prefix": dict(prefix_len=r.integers(0, s + 1, b).astype(np.int32)),
        "docs": dict(doc_ids=_docs(b, s, 3, seed)),
        "docs-full": dict(doc_ids=_docs(b, s, 2, seed + 1), causal=False),
        "docs-prefix-window": dict(doc_ids=_docs(b, s, 3, seed), prefix_len=r.integers(0, s + 1, b).astype(np.int32),
                                   window=max(3, s // 2)),
    }


def _gpu_ranges(b, s, mask):
    dev = {n: torch.from_numpy(x).cuda() if isinstance(x, np.ndarray) else x for n, x in mask.items()}
    return tp.attention_key_ranges(b, s, device="cuda", **dev)


# ------------------------------------------------------------------------- key ranges

@pytest.mark.parametrize("s", [1, 2, 7, 64, 300, 1000])
@pytest.mark.parametrize("name", list(_masks(2, 64)))
def test_key_ranges(name, s):
    mask = _masks(3, s, seed=s)[name]
    got = _gpu_ranges(3, s, mask).cpu().numpy()
    assert np.array_equal(got, oma.key_ranges(3, s, **mask))


@pytest.mark.parametrize("s", [8191, 8192, 8193, 20000, 32768, 32769, 70000])
def test_key_ranges_over_several_tiles(s):
    ids = np.sort(np.random.default_rng(s).integers(0, 9, (2, s)).astype(np.int32), axis=1)
    ids[0, : s // 2] = 4                                  # one document over more than a tile
    ids[1, s - 5:] = -7
    got = tp.attention_key_ranges(2, s, torch.from_numpy(ids).cuda(), causal=False).cpu().numpy()
    for bi in range(2):
        new = np.flatnonzero(np.concatenate([[True], ids[bi, 1:] != ids[bi, :-1]]))
        n = np.searchsorted(new, np.arange(s), side="right") - 1
        lo, hi = new[n], np.append(new, s)[n + 1]
        dead = ids[bi] < 0
        assert np.array_equal(got[bi, :, 0], np.where(dead, 0, lo)) and np.array_equal(got[bi, :, 1], np.where(dead, 0, hi))


def test_key_ranges_unsorted_ids_and_far_prefix():
    ids = np.array([[5, 5, 2, 2, 5, -1, -1, 5, 5, 0]], np.int32)     # a document is a run, not an id
    mask = dict(doc_ids=ids, prefix_len=np.array([2 ** 31 - 1], np.int32))
    assert np.array_equal(_gpu_ranges(1, 10, mask).cpu().numpy(), oma.key_ranges(1, 10, **mask))
    mask = dict(prefix_len=np.array([-4], np.int32), window=2 ** 40)
    assert np.array_equal(_gpu_ranges(1, 10, mask).cpu().numpy(), oma.key_ranges(1, 10, window=0))


# ------------------------------------------------------------------------- attention

@pytest.mark.parametrize("name", list(_masks(2, 64)))
@pytest.mark.parametrize("s", [200, 385])
def test_masks(name, s):
    mask = _masks(2, s, seed=s)[name]
    q, k, v, dO = _draw(s, 2, s, 2, 1, 64)
    ranges = oma.key_ranges(2, s, **mask)
    assert np.array_equal(_gpu_ranges(2, s, mask).cpu().numpy(), ranges)
    _check(q, k, v, dO, ranges)


@pytest.mark.parametrize("s", [1, 2, 63, 64, 65, 127, 128, 129, 255, 256, 257, 300, 513])
@pytest.mark.parametrize("hd", [64, 128])
def test_lengths(s, hd):
    q, k, v, dO = _draw(s + hd, 1, s, 2, 2, hd, "packed")
    _check(q, k, v, dO, oma.key_ranges(1, s))


@pytest.mark.parametrize("hd", [8, 16, 24, 40, 56, 72, 80, 96, 120])
@pytest.mark.parametrize("cap", [0.0, 20.0])
def test_head_widths(hd, cap):
    q, k, v, dO = _draw(hd, 2, 150, 4, 2, hd, "joined")
    _check(q, k, v, dO, oma.key_ranges(2, 150), cap=cap)


@pytest.mark.parametrize("heads,kv", [(1, 1), (6, 6), (6, 3), (8, 1), (5, 1), (16, 2)])
def test_grouped_heads(heads, kv):
    q, k, v, dO = _draw(heads * 10 + kv, 2, 140, heads, kv, 32, "joined")
    _check(q, k, v, dO, oma.key_ranges(2, 140), slopes=[2.0 ** -(h + 1) for h in range(heads)])


@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("cap,bias", [(5.0, False), (50.0, False), (0.0, True), (30.0, True)])
def test_caps_and_biases(hd, cap, bias):
    q, k, v, dO = _draw(hd, 1, 270, 2, 1, hd, std=2.0)
    slopes = [0.5, 0.03] if bias else None
    _check(q, k, v, dO, oma.key_ranges(1, 270, causal=False), cap=cap, slopes=slopes)
    _check(q, k, v, dO, oma.key_ranges(1, 270, window=100), cap=cap, slopes=slopes)


def test_negative_and_zero_slopes_and_another_scale():
    q, k, v, dO = _draw(3, 1, 190, 2, 2, 64)
    _check(q, k, v, dO, oma.key_ranges(1, 190), slopes=[-0.01, 0.0], scale=0.3)


def test_scores_far_apart():
    # a row's maximum grows by far more than the exponent's range from tile to tile, and falls again
    q, k, v, dO = _draw(5, 1, 520, 1, 1, 64)
    k = (k.float() * torch.linspace(0.1, 40, 520, device="cuda")[None, :, None, None]).bfloat16()
    _check(q, k, v, dO, oma.key_ranges(1, 520, causal=False), backward=False)
    _check(q, k.flip(1), v, dO, oma.key_ranges(1, 520, causal=False), backward=False)
    _check(q, k, v, dO, oma.key_ranges(1, 520), cap=30.0)


@pytest.mark.parametrize("seed", [0, 1])
def test_arbitrary_intervals(seed):
    # no order between neighbours, empty rows among them, ends outside the sequence
    s = 333
    r = np.random.default_rng(seed)
    ranges = np.sort(r.integers(-40, s + 40, (2, s, 2)), axis=2).astype(np.int32)
    ranges[:, r.integers(0, s, 60)] = 0
    ranges[0, 130:262] = [7, 7]                            # a whole block of rows without keys
    ranges[1, 5] = [200, 100]
    ranges[1, 6] = [-2 ** 31, 2 ** 31 - 1]
    q, k, v, dO = _draw(seed, 2, s, 2, 1, 64)
    _check(q, k, v, dO, ranges)


def test_nothing_visible():
    q, k, v, dO = _draw(1, 1, 150, 2, 2, 64)
    o, lse, dq, dk, dv = _check(q, k, v, dO, np.zeros((1, 150, 2), np.int32))
    assert torch.isneginf(lse).all()
    for t in (o, dq, dk, dv):
        assert torch.count_nonzero(t) == 0


def test_masked_keys_do_not_matter():
    # large finite values behind the mask, and in padding rows, change no bit
    s = 300
    q, k, v, dO = _draw(11, 1, s, 2, 2, 64)
    ids = np.full((1, s), -1, np.int32)
    ids[0, :100], ids[0, 100:250] = 1, 2
    ranges = _gpu_ranges(1, s, dict(doc_ids=ids))

    def run():
        o, lse = tp.masked_attention_forward(q, k, v, ranges)
        return (o, lse) + tp.masked_attention_backward(q, k, v, ranges, o, lse, dO)

    first = run()
    for t in (q, k, v, dO):
        t[:, 250:] = 1e4
    for a, b in zip(first, run()):
        assert torch.equal(a, b)
    assert torch.count_nonzero(first[0][:, 250:]) == 0


def test_empty_batch():
    q = torch.empty(0, 16, 2, 64, dtype=torch.bfloat16, device="cuda")
    ranges = tp.attention_key_ranges(0, 16, device="cuda")
    o, lse = tp.masked_attention_forward(q, q, q, ranges)
    dq, dk, dv = tp.masked_attention_backward(q, q, q, ranges, o, lse, q)
    assert ranges.shape == (0, 16, 2) and o.shape == q.shape and lse.shape == (0, 2, 16) and dq.shape == dk.shape == q.shape


def test_longer_rows_and_many_heads():
    q, k, v, dO = _draw(2, 1, 1500, 2, 1, 128, "joined")
    ids = np.zeros((1, 1500), np.int32)
    ids[0, 700:] = 1
    _check(q, k, v, dO, oma.key_ranges(1, 1500, doc_ids=ids), cap=40.0)


@pytest.mark.parametrize("hd", [64, 128])
def test_more_pieces_than_resident_ctas(hd):
    # 480 tiles of queries and 240 of keys, long and short ones mixed, on at most a CTA per SM
    b, s, heads, kv = 20, 140, 12, 6
    q, k, v, dO = _draw(hd, b, s, heads, kv, hd, "joined")
    ids = _docs(b, s, 4, 5)
    ids[3] = -1                                            # a sequence of padding alone
    _check(q, k, v, dO, oma.key_ranges(b, s, doc_ids=ids))


@pytest.mark.parametrize("hd,std,cap", [(64, 4.0, 3.0), (64, 1.0, 10.0), (128, 0.3, 100.0), (128, 1.0, 9.0),
                                        (128, 3.0, 20.0)])
def test_both_ways_of_the_cap(hd, std, cap):
    # scores far past the cap, scores that it hardly bends, and tiles of either kind in one call
    q, k, v, dO = _draw(hd + 1, 1, 300, 2, 1, hd, std=std)
    if cap == 20.0:
        k[:, :128] *= 0.05
    _check(q, k, v, dO, oma.key_ranges(1, 300), cap=cap)


@pytest.mark.parametrize("cap", [0.0, 20.0])
@pytest.mark.parametrize("hd,causal,window", [(64, True, 0), (64, False, 0), (128, True, 150), (128, False, 150), (40, False, 1)])
def test_steep_and_rising_slopes(hd, causal, window, cap):
    # slopes that raise a row's maximum from tile to tile, and one that favours far keys
    q, k, v, dO = _draw(hd + window, 1, 450, 4, 2, hd)
    _check(q, k, v, dO, oma.key_ranges(1, 450, causal=causal, window=window), cap=cap, slopes=[3.0, 0.4, 0.0, -0.02])


@pytest.mark.parametrize("scale", [1e-30, 1e-12, 30.0])
@pytest.mark.parametrize("cap", [0.0, 1e-6, 1e9])
def test_scales_out_of_the_ordinary(scale, cap):
    # where a cap's polynomial would leave fp32 it is not used
    q, k, v, dO = _draw(5, 1, 140, 2, 1, 64)
    ranges = oma.key_ranges(1, 140)
    lse = _check(q, k, v, dO, ranges, cap=cap, scale=scale, backward=scale < 1)[1]
    if cap == 1e9:   # a cap that no score comes near changes nothing: x^2 / 3 < 1e-11
        free = tp.masked_attention_forward(q, k, v, torch.from_numpy(ranges).cuda(), scale=scale)[1]
        assert ((lse - free).abs() <= 2.0 ** -20 * (1 + free.abs())).all()


def test_two_calls_at_once():
    # two streams, each with its own tensors and workspaces, in flight together
    sets = [_draw(20 + n, 2, 700, 8, 4, 128 if n else 64) for n in range(2)]
    ranges = tp.attention_key_ranges(2, 700, device="cuda")

    def step(t, stream=None):
        o, lse = tp.masked_attention_forward(t[0], t[1], t[2], ranges, stream=stream)
        return (o, lse) + tp.masked_attention_backward(t[0], t[1], t[2], ranges, o, lse, t[3], stream=stream)

    want = [step(t) for t in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    got = [[step(t, st) for t, st in zip(sets, streams)] for _ in range(3)]
    torch.cuda.synchronize()
    tp.tpmlp_device_status()
    for run in got:
        for a, b in zip(want, run):
            for x, y in zip(a, b):
                assert torch.equal(x, y)


def test_two_graphs_of_one_step():
    # each graph holds its own workspace; replayed in turn and with other inputs in between
    q, k, v, dO = _draw(30, 1, 390, 4, 4, 64)
    ranges = tp.attention_key_ranges(1, 390, device="cuda")
    graphs, outs = [], []
    tp.masked_attention_backward(q, k, v, ranges, *tp.masked_attention_forward(q, k, v, ranges), dO)
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            o, lse = tp.masked_attention_forward(q, k, v, ranges)
            outs.append((o, lse) + tp.masked_attention_backward(q, k, v, ranges, o, lse, dO))
        graphs.append(g)
    first = q.clone()
    q.mul_(-0.5)
    graphs[0].replay()
    other = [t.clone() for t in outs[0]]
    q.copy_(first)
    graphs[1].replay()
    graphs[0].replay()
    torch.cuda.synchronize()
    for a, b, c in zip(outs[0], outs[1], other):
        assert torch.equal(a, b)
    assert not torch.equal(outs[0][0], other[0])


def test_same_inputs_same_bits():
    q, k, v, dO = _draw(4, 2, 500, 8, 2, 64)
    ranges = tp.attention_key_ranges(2, 500, device="cuda")
    runs = []
    for _ in range(3):
        o, lse = tp.masked_attention_forward(q, k, v, ranges, softcap=30.0)
        runs.append((o, lse) + tp.masked_attention_backward(q, k, v, ranges, o, lse, dO, softcap=30.0))
    for other in runs[1:]:
        for a, b in zip(runs[0], other):
            assert torch.equal(a, b)


def test_gradients_against_differences():
    # the loss sum(o dO) in 64 bits, moved along random directions of q, k and v, against the kernel's gradients:
    # off by what the elements' tolerances allow
    q, k, v, dO = _draw(6, 1, 90, 2, 1, 64)
    ranges = oma.key_ranges(1, 90, window=40)
    sl, cap = [0.02, 0.1], 10.0
    _, _, dq, dk, dv = _check(q, k, v, dO, ranges, cap=cap, slopes=sl)
    r = np.random.default_rng(0)
    args = [_np(q), _np(k), _np(v)]
    f = oma.attention(*args, ranges, 0.125, cap, sl, _np(dO))
    for n, (g, name) in enumerate(((dq, "dq"), (dk, "dk"), (dv, "dv"))):
        d = r.standard_normal(args[n].shape)
        ends = []
        for h in (1e-5, -1e-5):
            moved = list(args)
            moved[n] = args[n] + h * d
            ends.append((oma.attention(*moved, ranges, 0.125, cap, sl)["o"] * _np(dO)).sum())
        slope = (ends[0] - ends[1]) / 2e-5
        each = (U * (f["dv_abs"] + np.abs(f["dv"])) + SLACK * f["dv_abs"] if name == "dv" else
                U * (f[name + "_d"] + f[name + "_abs"] + np.abs(f[name])) + SLACK * f[name + "_p"])
        assert abs((_np(g) * d).sum() - slope) <= (each * np.abs(d)).sum()
        assert abs((f[name] * d).sum() - slope) <= 1e-5 * (1 + abs(slope))


def test_graph_replays_and_other_stream():
    q, k, v, dO = _draw(8, 1, 260, 4, 2, 128)
    ranges = tp.attention_key_ranges(1, 260, device="cuda")

    def step(stream=None):
        o, lse = tp.masked_attention_forward(q, k, v, ranges, stream=stream)
        return (o, lse) + tp.masked_attention_backward(q, k, v, ranges, o, lse, dO, stream=stream)

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
    for _ in range(2):
        for t in held:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(want, held):
            assert torch.equal(a, b)
    tp.tpmlp_device_status()


def test_outputs_into_strided_views_leave_the_rest():
    b, s, heads, hd = 2, 77, 3, 40
    q, k, v, dO = _draw(9, b, s, heads, heads, hd, "packed")
    ranges = tp.attention_key_ranges(b, s, device="cuda")
    o, lse = tp.masked_attention_forward(q, k, v, ranges)
    want = (o,) + tp.masked_attention_backward(q, k, v, ranges, o, lse, dO)
    wide = [torch.full((b, s, heads, 3, hd + 8), 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    views = [wide[0][:, :, :, n, :hd] for n in range(3)]
    ov = wide[1][:, :, :, 1, :hd]
    tp.masked_attention_forward(q, k, v, ranges, o=ov)
    ov2 = wide[1][:, :, :, 1, :hd]
    dv2 = torch.full_like(wide[1], 7.0)[:, :, :, 1, :hd]
    dv2.copy_(dO)
    tp.masked_attention_backward(q, k, v, ranges, ov2, lse, dv2, dq=views[0], dk=views[1], dv=views[2])
    torch.cuda.synchronize()
    for a, x in zip(want, [ov] + views):
        assert torch.equal(a, x)
    assert (wide[0][..., hd:] == 7).all() and (wide[1][..., hd:] == 7).all() and (wide[1][:, :, :, 0] == 7).all()


def test_offsets_past_32_bits():
    # token rows of 128 KB: the last rows lie 5 GB behind the first, past 2^32 bytes and 2^31 elements
    s, ld, hd = 40000, 65536, 64
    big = torch.empty(s, ld, dtype=torch.bfloat16, device="cuda")
    gen = torch.Generator("cuda").manual_seed(3)
    big[:, :5 * hd] = torch.randn(s, 5 * hd, generator=gen, device="cuda").bfloat16()
    q, k, v, dO = (big[:, n * hd:(n + 1) * hd].view(1, s, 1, hd) for n in range(4))
    o = big[:, ld - hd:].view(1, s, 1, hd)
    ranges = tp.attention_key_ranges(1, s, window=50, device="cuda")
    _, lse = tp.masked_attention_forward(q, k, v, ranges, o=o)
    dq, dk, dv = (torch.empty(s, hd, dtype=torch.bfloat16, device="cuda").view(1, s, 1, hd) for _ in range(3))
    tp.masked_attention_backward(q, k, v, ranges, o, lse, dO, dq=dq, dk=dk, dv=dv)
    torch.cuda.synchronize()
    tail = slice(s - 300, s)                                # the last 300 rows alone, as a sequence of their own
    sub = [t[:, tail].clone() for t in (q, k, v, dO)]
    ranges2 = oma.key_ranges(1, 300, window=50)
    f = oma.attention(*(_np(t) for t in sub[:3]), ranges2, 0.125, dO=_np(sub[3]))
    _hold("o", o[:, tail][:, 50:], f["o"][:, 50:], (U * (f["o_abs"] + np.abs(f["o"])) + SLACK * f["o_abs"])[:, 50:])
    for name, g in (("dq", dq), ("dk", dk)):
        tol = U * (f[name + "_d"] + f[name + "_abs"] + np.abs(f[name])) + SLACK * f[name + "_p"]
        _hold(name, g[:, tail][:, 50:], f[name][:, 50:], tol[:, 50:])


# ------------------------------------------------------------------------- the operators in a row

@pytest.mark.parametrize("hd,style", [(64, "half"), (128, "interleaved")])
def test_norm_rotation_and_attention_together(hd, style):
    """One layer's attention as a model runs it, out of the packed QKV matrix and back into its gradient: each
    operator's output feeds the next, and each is held to the oracle on the very values that it was given."""
    b, s, heads = 2, 130, 3
    gen = torch.Generator("cuda").manual_seed(hd)
    qkv = torch.randn(b, s, heads, 3, hd, generator=gen, device="cuda").bfloat16()
    dO = torch.randn(b, s, heads, hd, generator=gen, device="cuda").bfloat16()
    gq, gk = (1 + 0.2 * torch.randn(hd, generator=gen, device="cuda") for _ in range(2))
    cos, sin = tp.rope_tables(4096, hd, device="cuda")
    pos = (torch.arange(s, device="cuda", dtype=torch.int32) + torch.tensor([[0], [3900]], device="cuda")).int().contiguous()
    ids = torch.zeros(b, s, dtype=torch.int32, device="cuda")
    ids[0, 60:], ids[1, 100:] = 1, -1
    pos[1, 100:] = -1
    ranges = tp.attention_key_ranges(b, s, doc_ids=ids)
    qn, kn = tp.qk_norm_rope(qkv[..., 0, :], qkv[..., 1, :], gq, gk, cos, sin, positions=pos, style=style)
    o, lse = tp.masked_attention_forward(qn, kn, qkv[..., 2, :], ranges, softcap=25.0)
    dqkv = torch.empty_like(qkv)
    dqn, dkn, _ = tp.masked_attention_backward(qn, kn, qkv[..., 2, :], ranges, o, lse, dO, softcap=25.0,
                                               dv=dqkv[..., 2, :])
    _, _, dgq, dgk = tp.qk_norm_rope_backward(qkv[..., 0, :], qkv[..., 1, :], gq, gk, cos, sin, dqn, dkn, positions=pos,
                                              style=style, dq=dqkv[..., 0, :], dk=dqkv[..., 1, :])
    torch.cuda.synchronize()
    tp.tpmlp_device_status()
    f = oma.attention(_np(qn), _np(kn), _np(qkv[..., 2, :]), ranges.cpu().numpy(), 1 / math.sqrt(hd), 25.0, None, _np(dO))
    _hold("o", o, f["o"], U * (f["o_abs"] + np.abs(f["o"])) + SLACK * f["o_abs"] + 1e-30)
    _hold("dv", dqkv[..., 2, :], f["dv"], U * (f["dv_abs"] + np.abs(f["dv"])) + SLACK * f["dv_abs"] + 1e-30)
    flat = pos.cpu().numpy().reshape(-1)
    c, sn = cos.cpu().numpy(), sin.cpu().numpy()
    for n, (y, dy, g, dg) in enumerate(((qn, dqn, gq, dgq), (kn, dkn, gk, dgk))):
        x = _np(qkv[..., n, :]).reshape(b * s, heads, hd)
        ref = oqr.forward(x, _np(g), 1e-5, c, sn, flat, style)
        _hold("y", y.reshape(b * s, heads, hd), ref, U * np.abs(ref) + 2.0 ** -18 * np.abs(ref).max(-1, keepdims=True) + 1e-30)
        dx, dgamma = oqr.backward(x, _np(g), 1e-5, c, sn, flat, style, _np(dy).reshape(b * s, heads, hd))
        _hold("dx", dqkv[..., n, :].reshape(b * s, heads, hd), dx,
              U * np.abs(dx) + 2.0 ** -16 * np.abs(dx).max(-1, keepdims=True) + 1e-30)
        _hold("dgamma", dg, dgamma, 2.0 ** -16 * (np.abs(_np(dy)).reshape(-1, hd).sum(0).max() + np.abs(dgamma)))
