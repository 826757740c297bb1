"""Masked attention on values at the ends of the number range: NaN, infinities and products past fp32 in visible
places. Most expectations are exact: a row that does not see the value keeps its bits."""
import math

import numpy as np
import pytest
import torch

import tensor_transformer_mlp_gb300 as tp
from oracle import masked_attention as oma
from test_gpu_masked_attention import _check, _draw

pytestmark = pytest.mark.gpu

U = 2.0 ** -8        # half a step of bf16
SLACK = 2.0 ** -12   # fp32 sums and exponents, 1/16 of it
S = 300
FORMS = [(64, 0.0, False), (64, 20.0, False), (64, 0.0, True), (128, 0.0, False), (128, 20.0, False), (128, 0.0, True),
         (128, 20.0, True)]


def _inputs(hd, seed=0):
    gen = torch.Generator("cuda").manual_seed(seed + hd)
    return [torch.randn(1, S, 2, hd, generator=gen, device="cuda").bfloat16() for _ in range(4)]


def _kw(cap, bias, **kw):
    return dict(softcap=cap, slopes=torch.tensor([0.02, 0.003], device="cuda") if bias else None, **kw)


def _forward(q, k, v, ranges, kw):
    out = tp.masked_attention_forward(q, k, v, ranges, **kw)
    torch.cuda.synchronize()
    tp.tpmlp_device_status()
    return out


@pytest.mark.parametrize("hd,cap,bias", FORMS)
def test_nan_in_a_query_or_key_reaches_the_rows_that_see_it(hd, cap, bias):
    q, k, v, _ = _inputs(hd)
    ranges = tp.attention_key_ranges(1, S, device="cuda")
    kw = _kw(cap, bias)
    o, lse = _forward(q, k, v, ranges, kw)
    bad = q.clone()
    bad[0, 140, 1, 3] = float("nan")
    o1, lse1 = _forward(bad, k, v, ranges, kw)
    assert torch.isnan(o1[0, 140, 1]).all() and torch.isnan(lse1[0, 1, 140])
    o1[0, 140, 1], lse1[0, 1, 140] = o[0, 140, 1], lse[0, 1, 140]
    assert torch.equal(o1, o) and torch.equal(lse1, lse)
    bad = k.clone()
    bad[0, 140, 0, 5] = float("nan")
    o1, lse1 = _forward(q, bad, v, ranges, kw)
    assert torch.isnan(o1[0, 140:, 0]).all() and torch.isnan(lse1[0, 0, 140:]).all()
    assert torch.equal(o1[:, :140], o[:, :140]) and torch.equal(lse1[:, :, :140], lse[:, :, :140])
    assert torch.equal(o1[:, :, 1], o[:, :, 1]) and torch.equal(lse1[:, 1], lse[:, 1])


@pytest.mark.parametrize("hd,cap,bias", FORMS)
def test_all_scores_nan(hd, cap, bias):
    # the maximum of such a row stays at its start
    q, k, v, _ = _inputs(hd)
    q[0, 7] = float("nan")
    o, lse = _forward(q, k, v, tp.attention_key_ranges(1, S, device="cuda"), _kw(cap, bias))
    assert torch.isnan(o[0, 7]).all() and torch.isnan(lse[0, :, 7]).all()
    o[0, 7], lse[0, :, 7] = 0, 0
    assert torch.isfinite(o).all() and torch.isfinite(lse).all()


@pytest.mark.parametrize("hd,cap,bias", FORMS)
def test_values_that_are_no_numbers(hd, cap, bias):
    q, k, v, _ = _inputs(hd)
    ranges = tp.attention_key_ranges(1, S, causal=False, device="cuda")
    kw = _kw(cap, bias)
    o, lse = _forward(q, k, v, ranges, kw)
    bad = v.clone()
    bad[0, 200, 0, 3], bad[0, 9, 1, 4], bad[0, 290, 1, 5] = float("nan"), float("inf"), -float("inf")
    o1, lse1 = _forward(q, k, bad, ranges, kw)
    assert torch.isnan(o1[0, :, 0, 3]).all()
    assert (o1[0, :, 1, 4] == float("inf")).all() and (o1[0, :, 1, 5] == -float("inf")).all()
    o1[0, :, 0, 3], o1[0, :, 1, 4:6] = o[0, :, 0, 3], o[0, :, 1, 4:6]
    assert torch.equal(o1, o) and torch.equal(lse1, lse)


@pytest.mark.parametrize("how", ["infinite key", "product past fp32", "scale past fp32"])
@pytest.mark.parametrize("hd,cap,bias", FORMS)
def test_infinite_scores(hd, cap, bias, how):
    # key 150 scores +inf with one half of the queries and -inf with the other
    q, k, v, _ = _inputs(hd)
    sign = torch.where(torch.arange(S, device="cuda") % 3 == 0, 1.0, -1.0).bfloat16()
    scale = 1 / math.sqrt(hd)
    if how == "infinite key":
        q[:, :, :, 0] = sign[None, :, None]
        k[0, 150, :, 0] = float("inf")
    elif how == "product past fp32":
        q[:, :, :, 0] = sign[None, :, None] * 2.0 ** 66
        k[:, :, :, 0] = 0
        k[0, 150, :, 0] = 2.0 ** 66
    else:  # 2^32 as a product, finite; past fp32 with the scale; all other scores are zeros
        q.zero_(), k.zero_()
        q[:, :, :, 0] = sign[None, :, None] * 2.0 ** 16
        k[0, 150, :, 0] = 2.0 ** 16
        scale = 1e30
    ranges = tp.attention_key_ranges(1, S, causal=False, device="cuda")
    o, lse = _forward(q, k, v, ranges, _kw(cap, bias, scale=scale))
    i = torch.arange(S, device="cuda")
    for h in range(2):
        x = q[0, :, h].double() @ k[0, :, h].double().T
        x[x.abs() > 3.5e38] = x[x.abs() > 3.5e38].sign() * float("inf")
        x = x * scale
        x[x.abs() > 3.5e38] = x[x.abs() > 3.5e38].sign() * float("inf")
        y = cap * torch.tanh(x / cap) if cap else x
        if bias:
            y = y - [0.02, 0.003][h] * (i[:, None] - i).abs()
        p = torch.softmax(y, -1)                       # NaN in a row with +inf
        none = p.isnan().any(-1)
        assert bool(none.any()) == (cap == 0.0)
        assert torch.equal(o[0, :, h].isnan().all(-1), none) and torch.equal(lse[0, h].isnan(), none)
        p, vh = p[~none], v[0, :, h].double()
        tol = U * (p @ vh.abs() + (p @ vh).abs()) + SLACK * (p @ vh.abs())
        assert ((o[0, ~none, h].double() - p @ vh).abs() <= tol).all()
        want = torch.logsumexp(y[~none], -1)
        mag = (q[0, :, h].double().abs() @ k[0, :, h].double().abs().T * scale)[~none]
        mag = torch.where(mag > 1e6, 0.0, mag).amax(-1)  # where it counts scores are ordinary
        near = hd * 2.0 ** -24 * mag + 2.0 ** -20 * (1 + want.abs()) + 2.0 ** -21 * cap + 3 * 2.0 ** -24 * 256 * 0.02
        assert ((lse[0, h, ~none].double() - want).abs() <= near).all()


@pytest.mark.parametrize("hd", [64, 128])
def test_position_past_the_table_is_seen_in_the_loss(hd):
    # the norm with rotation writes NaN for it; no later row of the sequence may come out as a number
    q, k, v, _ = _inputs(hd)
    g = torch.ones(hd, device="cuda")
    cos, sin = tp.rope_tables(64, hd, device="cuda")
    pos = torch.full((1, S), 5, dtype=torch.int32, device="cuda")
    pos[0, 100] = 64
    qn, kn = tp.qk_norm_rope(q, k, g, g, cos, sin, positions=pos)
    o, lse = _forward(qn, kn, v, tp.attention_key_ranges(1, S, device="cuda"), {})
    assert torch.isnan(o[0, 100:]).all() and torch.isnan(lse[0, :, 100:]).all()
    assert torch.isfinite(o[0, :100]).all() and torch.isfinite(lse[0, :, :100]).all()
    assert np.isnan(o.float().sum().item())


@pytest.mark.parametrize("hd,bias", [(64, False), (64, True), (128, False), (128, True)])
def test_gradients_of_rows_whose_scores_are_all_minus_infinity(hd, bias):
    # such a row weighs nothing: every gradient has the bits that it has without the row
    q, k, v, dO = _inputs(hd)
    q[..., 0], k[..., 0] = 0, -2.0 ** 66
    rows = [7, 140, 141, 299]
    q[0, rows, :, 0] = 2.0 ** 66
    ranges = tp.attention_key_ranges(1, S, causal=False, device="cuda")
    none = ranges.clone()
    none[0, rows] = 0
    runs = []
    for r in (ranges, none):
        o, lse = _forward(q, k, v, r, _kw(0.0, bias))
        assert torch.isneginf(lse[:, :, rows]).all() and torch.count_nonzero(o[:, rows]) == 0
        runs.append((o, lse) + tp.masked_attention_backward(q, k, v, r, o, lse, dO, **_kw(0.0, bias)))
    torch.cuda.synchronize()
    tp.tpmlp_device_status()
    assert torch.count_nonzero(runs[0][2][:, rows]) == 0
    for a, b in zip(*runs):
        assert torch.equal(a, b)
    for t in runs[0][2:]:
        assert torch.isfinite(t).all()


CAPS = [(1e2, 90.0), (1e3, 3.0), (1e3, 200.0), (1e4, 100.0), (1e5, 100.0), (1e5, 1000.0), (1e6, 1000.0), (1e7, 1e4),
        (1e10, 1e4)]


@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("cap,most", CAPS)
def test_caps_far_above_the_scores(hd, cap, most):
    """A capped score is good relative to itself, not to the cap: tanh to 1.1e-6 of itself (its forms' 4.9e-7, or 2.6e-7 in
    absolute terms from |x| = 0.25 on), the roundings of its factors and of the row's statistics 2^-24 each: 2^-19 in all.
    The products q.k are sums of small whole numbers and carry no error."""
    gen = torch.Generator("cuda").manual_seed(hd)
    q, k = (torch.randint(-8, 9, (1, S, 2, hd), generator=gen, device="cuda").bfloat16() for _ in range(2))
    v, dO = (torch.randn(1, S, 2, hd, generator=gen, device="cuda").bfloat16() for _ in range(2))
    qd, kd, vd, gd = (t[0].double().transpose(0, 1) for t in (q, k, v, dO))
    whole = qd @ kd.transpose(1, 2)
    scale = float(np.float32(most / whole.abs().max().item()))
    ranges = tp.attention_key_ranges(1, S, causal=False, device="cuda")
    kw = dict(scale=scale, softcap=cap)
    o, lse = _forward(q, k, v, ranges, kw)
    dq, dk, dv = tp.masked_attention_backward(q, k, v, ranges, o, lse, dO, **kw)
    y = cap * torch.tanh(whole * scale / float(np.float32(cap)))
    want = torch.logsumexp(y, -1)
    assert ((lse[0].double() - want).abs() <= 2.0 ** -19 * y.abs().amax(-1) + 2.0 ** -20).all()
    free = tp.masked_attention_forward(q, k, v, ranges, scale=scale)[1][0]
    if most / cap <= 1e-3:  # the cap takes x^2 / 3 = 3e-7 of a score at most
        assert ((lse[0] - free).abs() <= 2.0 ** -20 * (1 + y.abs().amax(-1))).all()
    p = torch.softmax(y, -1)
    off = SLACK + 2 * 2.0 ** -19 * 2 * most   # P from a score and from lse
    gone = 300 * 8 * 2.0 ** -126              # a probability below 2^-126 is zero in fp32: 300 of them, |v| and |dO| below 8
    assert max(vd.abs().max(), gd.abs().max()) < 8
    for got, to, x in ((o, p, vd), (dv, p.transpose(1, 2), gd)):
        ref, size = to @ x, to @ x.abs()
        assert ((got[0].transpose(0, 1).double() - ref).abs() <= U * (size + ref.abs()) + off * size + gone).all()
    assert torch.isfinite(dq).all() and torch.isfinite(dk).all()


@pytest.mark.parametrize("hd", [64, 128])
def test_scores_of_2_to_the_29(hd):
    # whole products of unlike size lie 10^5 apart there: a row's output is the mean of the values of its largest
    gen = torch.Generator("cuda").manual_seed(hd + 1)
    q, k = (torch.randint(-8, 9, (1, S, 2, hd), generator=gen, device="cuda").bfloat16() for _ in range(2))
    v = torch.randn(1, S, 2, hd, generator=gen, device="cuda").bfloat16()
    qd, kd, vd = (t[0].double().transpose(0, 1) for t in (q, k, v))
    whole = qd @ kd.transpose(1, 2)
    scale = float(np.float32(2.0 ** 29 / whole.abs().max().item()))
    o, lse = _forward(q, k, v, tp.attention_key_ranges(1, S, causal=False, device="cuda"), dict(scale=scale))
    y = whole * scale
    p = torch.softmax(y, -1)
    assert ((lse[0].double() - torch.logsumexp(y, -1)).abs() <= 2.0 ** -21 * y.abs().amax(-1)).all()
    ref, size = p @ vd, p @ vd.abs()
    assert ((o[0].transpose(0, 1).double() - ref).abs() <= U * (size + ref.abs()) + SLACK * size).all()


def test_a_piece_of_work_longer_than_the_limit_of_a_wait():
    # one block of queries sees 402 million keys, which takes 3.6 s, past the 2 s that a wait may last without progress
    s, hd = 3 << 27, 8
    q = torch.zeros(1, s, 1, hd, dtype=torch.bfloat16, device="cuda")
    v = torch.ones_like(q)
    v[0, -1, 0, 0] = s / 2
    ranges = torch.zeros(1, s, 2, dtype=torch.int32, device="cuda")
    ranges[0, -256:, 1] = s
    ranges[0, 5, 1] = 6
    o, lse = tp.masked_attention_forward(q, q, v, ranges)
    torch.cuda.synchronize()
    tp.tpmlp_device_status()
    assert ((lse[0, 0, -256:] - math.log(s)).abs() < 1e-5).all()
    assert (o[0, -256:, 0, 0] > o[0, -256:, 0, 1]).all()          # the last key is among them
    assert torch.equal(o[0, 5, 0].float(), torch.ones(hd, device="cuda"))
    assert torch.count_nonzero(o[0, :, 0, 1]) == 257 and torch.isfinite(lse).sum() == 257


@pytest.mark.parametrize("cap,bias", [(0.0, False), (30.0, True)])
@pytest.mark.parametrize("hd", [64, 128])
def test_sums_over_a_million_rows(hd, cap, bias):
    """Sums of a million terms of one sign and size, in every accumulator: O and dQ of the last 128 queries over all keys,
    dK and dV of the first 64 keys over all queries. All scores are zero (queries and keys use different columns, the
    slopes are zero), so P is 2^-20 or 2^-6; the first column of V is 0 or 2 and that of dO 1, so dX is P or -P: no term is
    rounded. What is left is the result's rounding, and what an accumulator loses over the 2^15 rows that it holds at most:
    2^-26 of it a row, 2^-11 in all."""
    s, half = 1 << 20, hd // 2
    gen = torch.Generator("cuda").manual_seed(hd)
    rand = lambda: torch.rand(s, half, generator=gen, device="cuda").bfloat16()  # noqa: E731
    q, k, v, dO = (torch.zeros(1, s, 1, hd, dtype=torch.bfloat16, device="cuda") for _ in range(4))
    sign = torch.where(torch.arange(s, device="cuda") % 2 == 0, 1.0, -1.0)
    q[0, :, 0, :half] = rand()
    k[0, :, 0, half:] = rand() * sign[:, None].bfloat16()
    v[0, :, 0, 0] = 1 + sign
    v[0, :, 0, half:] = rand()
    dO[0, :, 0, 0] = 1
    dO[0, :, 0, 1:half] = rand()[:, 1:]
    ranges = torch.zeros(1, s, 2, dtype=torch.int32, device="cuda")
    ranges[0, :, 1] = 64
    ranges[0, -128:, 1] = s
    kw = dict(softcap=cap, slopes=torch.zeros(1, device="cuda") if bias else None, scale=0.25)
    o, lse = _forward(q, k, v, ranges, kw)
    dq, dk, dv = tp.masked_attention_backward(q, k, v, ranges, o, lse, dO, **kw)
    torch.cuda.synchronize()
    tp.tpmlp_device_status()
    assert (lse[0, 0, :-128] - math.log(64)).abs().max() < 1e-6 and (lse[0, 0, -128:] - math.log(s)).abs().max() < 4e-6
    qd, kd, vd, gd, sg = q[0, :, 0].double(), k[0, :, 0].double(), v[0, :, 0].double(), dO[0, :, 0].double(), sign.double()
    few, all_q, all_g = slice(0, 64), qd[-128:].sum(0) / s, gd[-128:].sum(0) / s
    want = {"o": vd.mean(0), "dq": 0.25 * (sg[:, None] * kd).mean(0),
            "dv": gd[:-128].sum(0) / 64 + all_g, "dk": 0.25 * (qd[:-128].sum(0) / 64 + all_q)}
    got = {"o": o[0, -128:, 0], "dq": dq[0, -128:, 0], "dv": dv[0, few, 0], "dk": dk[0, few, 0].double() * sg[few, None]}
    for name, w in want.items():
        off = (got[name].double() - w).abs()
        assert (off <= (U + 2.0 ** -11) * w.abs()).all(), (name, (off / w.abs().clamp(min=1e-30)).max().item())
    rest = (dv[0, 64:, 0].double() - all_g).abs() <= (U + 2.0 ** -11) * all_g.abs()
    assert rest.all()


@pytest.mark.parametrize("hd,cap,bias", [(64, 0.0, True), (128, 20.0, False)])
def test_keys_shared_by_many_heads(hd, cap, bias):
    # a key is seen by 17 tiles of 32 heads' queries: its sums are long though the sequence is not
    q, k, v, dO = _draw(hd, 1, 2100, 32, 1, hd, "joined")
    _check(q, k, v, dO, oma.key_ranges(1, 2100, causal=False), cap=cap, slopes=[2.0 ** -(4 + h / 8) for h in range(32)] if bias else None)


def test_a_long_row_whose_maximum_moves():
    # parts of O under maxima of their own, falling and rising, against 64 bits; some rows see the middle only
    s, hd = 70000, 64
    gen = torch.Generator("cuda").manual_seed(7)
    q, k, v = (torch.randn(1, s, 1, hd, generator=gen, device="cuda").bfloat16() for _ in range(3))
    q, k = q.abs(), k.abs() * torch.linspace(0.1, 3, s, device="cuda")[None, :, None, None].bfloat16()
    ranges = torch.zeros(1, s, 2, dtype=torch.int32, device="cuda")
    ranges[0, -200:, 1] = s
    ranges[0, -100:-50, 0], ranges[0, -100:-50, 1] = 33000, 65600
    for keys in (k, k.flip(1)):
        o, lse = _forward(q, keys, v, ranges, {})
        x = q[0, -200:, 0].double() @ keys[0, :, 0].double().T / 8
        j = torch.arange(s, device="cuda")
        x[(j < ranges[0, -200:, :1]) | (j >= ranges[0, -200:, 1:])] = -math.inf
        p, vd = torch.softmax(x, -1), v[0, :, 0].double()
        size = p @ vd.abs()
        assert ((o[0, -200:, 0].double() - p @ vd).abs() <= U * (size + (p @ vd).abs()) + SLACK * size).all()
        want = torch.logsumexp(x, -1)
        assert ((lse[0, 0, -200:].double() - want).abs() <= 2.0 ** -20 * (1 + want.abs()) + hd * 2.0 ** -24 * x.amax(-1)).all()


@pytest.mark.parametrize("causal", [True, False])
def test_windows_of_any_length(causal):
    # past 64 bits too, of which ctypes would pass the lower ones
    free = tp.attention_key_ranges(2, 40, causal=causal, device="cuda")
    for window in (40, 41, 2 ** 31, 2 ** 63 - 1, 2 ** 63, 2 ** 64, 2 ** 64 + 5):
        assert torch.equal(tp.attention_key_ranges(2, 40, causal=causal, window=window, device="cuda"), free)
    assert not torch.equal(tp.attention_key_ranges(2, 40, causal=causal, window=39, device="cuda"), free)
    for window in (-1, -2 ** 64, -2 ** 64 + 5):
        with pytest.raises(tp.TpmlpError, match="window must be >= 0"):
            tp.attention_key_ranges(2, 40, window=window, device="cuda")
    ids = torch.zeros(2, 40, dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError, match="not on cpu"):
        tp.attention_key_ranges(2, 40, doc_ids=ids, device="cpu")
    assert torch.equal(tp.attention_key_ranges(2, 40, doc_ids=ids, causal=causal, device="cuda"), free)
