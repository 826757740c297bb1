"""Host-side checks of the masked-attention and norm-with-rotation entry points, no GPU needed: every refusal comes
before anything touches a device. Also pins of their oracles to something other than themselves."""
import numpy as np
import pytest
import torch

from oracle import masked_attention as oma
from oracle import qk_norm_rope as oqr
from tensor_transformer_mlp_gb300 import _binding

OK, INVALID, SHAPE, DTYPE, ALIGN, CUDA, TIMEOUT, WORKSPACE = range(8)
F32, BF16 = 0, 1
FAKE = 0x10000  # never dereferenced: every call below fails validation first


@pytest.fixture(scope="module")
def lib():
    return _binding.load_library(build_if_missing=True)


# ------------------------------------------------------------------------- refusals

def test_key_range_refusals(lib):
    def call(ids=FAKE, prefix=None, causal=1, window=0, out=FAKE, b=2, s=16):
        return lib.tpmlp_attention_key_ranges(ids, prefix, causal, window, out, b, s, None)
    assert call(causal=2) == INVALID
    assert call(window=-1) == INVALID
    assert call(prefix=FAKE, causal=0) == INVALID       # everything is visible anyway
    assert call(out=None) == INVALID
    assert call(out=FAKE + 4) == ALIGN
    assert call(ids=FAKE + 2) == ALIGN
    assert call(prefix=FAKE + 1) == ALIGN
    assert call(b=-1) == SHAPE and call(s=-1) == SHAPE
    assert call(b=1 << 20, s=1 << 20) == SHAPE
    assert call(b=1, s=2 ** 31 - 1) == SHAPE and call(b=1, s=(1 << 30) + 1) == SHAPE
    assert call(b=0, out=None) == OK and call(s=0) == OK


def fwd(lib, q=FAKE, k=FAKE, v=FAKE, rng=FAKE, slopes=None, scale=0.1, cap=0.0, o=FAKE, lse=FAKE, b=2, s=16, heads=4,
        kv=2, hd=64, ldq=256, hsq=64, ldk=128, hsk=64, ldv=128, hsv=64, ldo=256, hso=64, dt=BF16):
    return lib.tpmlp_masked_attention_forward(q, k, v, rng, slopes, scale, cap, o, lse, b, s, heads, kv, hd, ldq, hsq,
                                              ldk, hsk, ldv, hsv, ldo, hso, dt, None)


def test_forward_refusals(lib):
    for name in ("q", "k", "v", "rng", "o", "lse"):
        assert fwd(lib, **{name: None}) == INVALID, name
    for name in ("q", "k", "v", "o"):
        assert fwd(lib, **{name: FAKE + 8}) == ALIGN, name
    assert fwd(lib, rng=FAKE + 4) == ALIGN and fwd(lib, lse=FAKE + 2) == ALIGN and fwd(lib, slopes=FAKE + 1) == ALIGN
    assert fwd(lib, dt=F32) == DTYPE and fwd(lib, dt=7) == DTYPE
    assert fwd(lib, kv=3) == SHAPE and fwd(lib, heads=0) == SHAPE and fwd(lib, kv=0) == SHAPE
    assert fwd(lib, hd=60) == SHAPE and fwd(lib, hd=136) == SHAPE and fwd(lib, hd=0) == SHAPE
    assert fwd(lib, b=-1) == SHAPE and fwd(lib, s=-1) == SHAPE and fwd(lib, b=1 << 16, s=1 << 16) == SHAPE
    assert fwd(lib, b=1, s=(1 << 30) + 1, ldq=8) == SHAPE and fwd(lib, b=65536, s=1) == SHAPE
    assert fwd(lib, heads=65536, kv=1) == SHAPE
    assert fwd(lib, b=1, s=1 << 20, ldk=1 << 20) == SHAPE    # a sequence's keys span 2^40 elements
    for name in ("ldq", "hsq", "ldk", "hsk", "ldv", "hsv", "ldo", "hso"):
        assert fwd(lib, **{name: 0}) == SHAPE, name      # a broadcast tensor
        assert fwd(lib, **{name: -64}) == SHAPE, name
        assert fwd(lib, **{name: 68}) == SHAPE, name
        assert fwd(lib, **{name: 1 << 50}) == SHAPE, name
    assert fwd(lib, ldo=128) == SHAPE                    # the output's heads of neighbouring tokens overlap
    assert fwd(lib, hso=56) == SHAPE
    for bad in (0.0, -1.0, float("inf"), float("nan")):
        assert fwd(lib, scale=bad) == INVALID
    for bad in (-1.0, float("inf"), float("nan")):
        assert fwd(lib, cap=bad) == INVALID
    assert fwd(lib, scale=2e30) == INVALID and fwd(lib, cap=2e30) == INVALID and fwd(lib, scale=1.0, cap=1e-38) == INVALID
    assert fwd(lib, b=65535, s=1, heads=65535, kv=1, ldq=65535 * 64, ldo=65535 * 64) == SHAPE   # 2^32 pieces of work
    assert fwd(lib, b=0, q=None) == OK and fwd(lib, s=0, o=None) == OK


def test_backward_refusals(lib):
    size = lib.tpmlp_masked_attention_backward_workspace_size(2, 16, 4)
    assert size >= 2 * 16 * 4 * 4 and lib.tpmlp_masked_attention_backward_workspace_size(0, 16, 4) == 0

    def bwd(ptrs=None, strides=None, ws=FAKE, wsb=size, dt=BF16, b=2, s=16):
        p = dict(q=FAKE, k=FAKE, v=FAKE, rng=FAKE, slopes=None, o=FAKE, lse=FAKE, do=FAKE, dq=FAKE, dk=FAKE, dv=FAKE)
        p.update(ptrs or {})
        st = dict(ldq=256, hsq=64, ldk=128, hsk=64, ldv=128, hsv=64, ldo=256, hso=64, lddq=256, hsdq=64, lddk=128,
                  hsdk=64, lddv=128, hsdv=64)
        st.update(strides or {})
        return lib.tpmlp_masked_attention_backward(p["q"], p["k"], p["v"], p["rng"], p["slopes"], 0.1, 0.0, p["o"],
                                                   p["lse"], p["do"], p["dq"], p["dk"], p["dv"], b, s, 4, 2, 64,
                                                   *st.values(), dt, ws, wsb, None)
    for name in ("q", "k", "v", "rng", "o", "lse", "do", "dq", "dk", "dv"):
        assert bwd({name: None}) == INVALID, name
    for name in ("q", "k", "v", "o", "do", "dq", "dk", "dv"):
        assert bwd({name: FAKE + 8}) == ALIGN, name
    for name in ("lddq", "hsdq", "lddk", "hsdk", "lddv", "hsdv"):
        assert bwd(strides={name: 0}) == SHAPE and bwd(strides={name: 12}) == SHAPE, name
    assert bwd(strides={"lddk": 64}) == SHAPE and bwd(strides={"hsdv": 48}) == SHAPE
    assert bwd(ws=None) == WORKSPACE and bwd(wsb=size - 1) == WORKSPACE and bwd(ws=FAKE + 128) == ALIGN
    assert bwd(dt=F32) == DTYPE
    assert bwd(b=0, ws=None) == OK


def test_rope_refusals(lib):
    def call(q=FAKE, k=FAKE, gq=FAKE, gk=FAKE, eps=1e-5, cos=FAKE, sin=FAKE, pos=None, table=8, rot=64, style=0, qo=FAKE,
             ko=FAKE, b=1, s=8, heads=4, kv=2, hd=64, strides=(256, 64, 128, 64, 256, 64, 128, 64), dt=BF16):
        return lib.tpmlp_qk_norm_rope(q, k, gq, gk, eps, cos, sin, pos, table, rot, style, qo, ko, b, s, heads, kv, hd,
                                      *strides, dt, None)
    for name in ("q", "k", "gq", "gk", "cos", "sin", "qo", "ko"):
        assert call(**{name: None}) == INVALID, name
    for name in ("q", "k", "qo", "ko"):
        assert call(**{name: FAKE + 8}) == ALIGN, name
    for name in ("gq", "gk", "cos", "sin", "pos"):
        assert call(**{name: FAKE + 2}) == ALIGN, name
    assert call(dt=3) == DTYPE and call(style=2) == INVALID
    assert call(eps=0.0) == INVALID and call(eps=float("nan")) == INVALID
    assert call(rot=63) == SHAPE and call(rot=0) == SHAPE and call(rot=66) == SHAPE
    assert call(hd=60) == SHAPE and call(hd=264) == SHAPE and call(table=0) == SHAPE
    assert call(b=-1) == SHAPE and call(heads=0) == SHAPE and call(b=1 << 16, s=1 << 16) == SHAPE
    good = (256, 64, 128, 64, 256, 64, 128, 64)
    for n in range(8):
        assert call(strides=good[:n] + (0,) + good[n + 1:]) == SHAPE
        assert call(strides=good[:n] + (1 << 50,) + good[n + 1:]) == SHAPE
    assert call(strides=good[:4] + (192,) + good[5:]) == SHAPE      # overlapping outputs
    assert call(b=0, q=None) == OK

    def back(ws=FAKE, wsb=1 << 20, dgq=FAKE, dq=FAKE, strides=good + good[4:], b=1):
        return lib.tpmlp_qk_norm_rope_backward(FAKE, FAKE, FAKE, FAKE, 1e-5, FAKE, FAKE, None, 8, 64, 0, FAKE, FAKE, dq,
                                               FAKE, dgq, FAKE, b, 8, 4, 2, 64, *strides, BF16, ws, wsb, None)
    need = lib.tpmlp_qk_norm_rope_backward_workspace_size(1, 8, 64)
    assert need == 1024 * 64 * 4 and lib.tpmlp_qk_norm_rope_backward_workspace_size(0, 8, 64) == 0
    assert back(ws=None) == WORKSPACE and back(wsb=need - 1) == WORKSPACE and back(ws=FAKE + 8) == ALIGN
    assert back(dgq=None) == INVALID and back(dq=None) == INVALID
    assert back(strides=good + (256, 64, 64, 64)) == SHAPE


def test_outputs_that_are_inputs_are_refused(lib):
    at = [FAKE + 4096 * n for n in range(12)]
    good = (256, 64, 128, 64, 256, 64, 128, 64)

    def forward(**kw):
        ptrs = dict(q=at[0], k=at[1], v=at[2], rng=at[3], o=at[4], lse=at[5])
        return fwd(lib, **{**ptrs, **kw})
    for name in ("q", "k", "v"):
        assert forward(o=dict(q=at[0], k=at[1], v=at[2])[name]) == INVALID, name
    assert forward(lse=at[4]) == INVALID and forward(lse=at[3]) == INVALID and forward(slopes=at[5]) == INVALID

    size = lib.tpmlp_masked_attention_backward_workspace_size(2, 16, 4)

    def backward(dq=at[6], dk=at[7], dv=at[8], ws=at[9]):
        return lib.tpmlp_masked_attention_backward(at[0], at[1], at[2], at[3], None, 0.1, 0.0, at[4], at[5], at[10], dq, dk,
                                                   dv, 2, 16, 4, 2, 64, *(good[:4] + good[2:4] + good[:2] + good[:4]
                                                                          + good[2:4]), BF16, ws, size, None)
    assert backward(dq=at[0]) == INVALID and backward(dq=at[10]) == INVALID and backward(dk=at[8]) == INVALID
    assert backward(dv=at[2]) == INVALID and backward(ws=at[5]) == INVALID

    def rope(qo=at[8], ko=at[9], strides=good):
        return lib.tpmlp_qk_norm_rope(at[0], at[1], at[2], at[3], 1e-5, at[4], at[5], None, 8, 64, 0, qo, ko, 1, 8, 4, 2, 64,
                                      *strides, BF16, None)
    assert rope(qo=at[1]) == INVALID and rope(ko=at[0]) == INVALID and rope(qo=at[9]) == INVALID and rope(ko=at[2]) == INVALID
    assert rope(qo=at[0], strides=good[:4] + (512, 64, 128, 64)) == INVALID    # in place, but elsewhere

    def rope_back(dq=at[8], dk=at[9], dgq=at[10], ws=at[11], strides=good + good[4:]):
        return lib.tpmlp_qk_norm_rope_backward(at[0], at[1], at[2], at[3], 1e-5, at[4], at[5], None, 8, 64, 0, at[6], at[7],
                                               dq, dk, dgq, at[10] + 2048, 1, 8, 4, 2, 64, *strides, BF16, ws, 1 << 20, None)
    assert rope_back(dq=at[1]) == INVALID and rope_back(dk=at[6]) == INVALID and rope_back(dq=at[9]) == INVALID
    assert rope_back(dgq=at[2]) == INVALID and rope_back(ws=at[8]) == INVALID
    assert rope_back(dq=at[6], strides=good + (512, 64, 128, 64)) == INVALID


def test_binding_refuses_what_the_library_cannot_see():
    import tensor_transformer_mlp_gb300 as tp
    q = torch.zeros(1, 8, 2, 64, dtype=torch.bfloat16)
    r = torch.zeros(1, 8, 2, dtype=torch.int32)
    with pytest.raises(ValueError):                         # not on a GPU
        tp.masked_attention_forward(q, q, q, r)
    with pytest.raises(ValueError):
        tp.attention_key_ranges(1, 8, device="cpu")
    with pytest.raises(ValueError):                         # ranges of another shape or type
        tp.masked_attention_forward(q, q, q, r[:, :4])
    with pytest.raises(ValueError):
        tp.masked_attention_forward(q, q, q, r.long())
    with pytest.raises(ValueError):                         # [b, heads, s, hd] memory: no one token stride
        t = torch.zeros(2, 2, 8, 64, dtype=torch.bfloat16).transpose(1, 2)
        tp.masked_attention_forward(t, t, t, torch.zeros(2, 8, 2, dtype=torch.int32))
    with pytest.raises(ValueError):                         # columns not contiguous
        t = torch.zeros(1, 8, 64, 2, dtype=torch.bfloat16).transpose(2, 3)
        tp.masked_attention_forward(t, t, t, r)
    with pytest.raises(ValueError):
        tp.masked_attention_forward(q, q.float(), q, r)
    with pytest.raises(ValueError):
        tp.attention_key_ranges(1, 8, doc_ids=torch.zeros(1, 7, dtype=torch.int32))
    with pytest.raises(ValueError):                         # a table of no rows and columns
        tp.qk_norm_rope(q, q, torch.ones(64), torch.ones(64), torch.ones(64), torch.ones(64))


# ------------------------------------------------------------------------- the oracles' pins

@pytest.mark.parametrize("cap,bias", [(0.0, False), (7.0, True)])
def test_attention_oracle_against_autograd(cap, bias):
    r = np.random.default_rng(0)
    b, s, heads, kv, hd = 2, 17, 4, 2, 8
    q, k, v, dO = (r.standard_normal((b, s, n, hd)) for n in (heads, kv, kv, heads))
    ids = np.array([[0] * 9 + [1] * 8, [3] * 12 + [-1] * 5])
    ranges = oma.key_ranges(b, s, doc_ids=ids)
    slopes = [0.3, 0.1, 0.02, 0.0] if bias else None
    f = oma.attention(q, k, v, ranges, 0.4, cap, slopes, dO)
    tq, tk, tv = (torch.tensor(x, requires_grad=True) for x in (q, k, v))
    y = torch.einsum("bihd,bjhd->bhij", tq, tk.repeat_interleave(2, 2)) * 0.4
    if cap:
        y = cap * torch.tanh(y / cap)
    i = torch.arange(s)
    if bias:
        y = y - torch.tensor(slopes, dtype=torch.float64).view(1, -1, 1, 1) * (i[:, None] - i).abs()
    doc = torch.tensor(ids)
    seen = (doc[:, :, None] == doc[:, None]) & (doc[:, :, None] >= 0) & (i[:, None] >= i)
    live = seen.any(-1)
    y = y.masked_fill(~seen[:, None], -1e300)
    P = torch.softmax(y, -1) * live[:, None, :, None]
    o = torch.einsum("bhij,bjhd->bihd", P, tv.repeat_interleave(2, 2))
    o.backward(torch.tensor(dO))
    for name, got in (("o", o), ("dq", tq.grad), ("dk", tk.grad), ("dv", tv.grad)):
        assert np.abs(f[name] - got.detach().numpy()).max() < 1e-12, name
    lse = torch.logsumexp(y, -1).detach().numpy()
    assert np.array_equal(np.isneginf(f["lse"]), np.broadcast_to(~live.numpy()[:, None], lse.shape))
    keep = np.isfinite(f["lse"])
    assert np.abs((f["lse"] - lse)[keep]).max() < 1e-12


@pytest.mark.parametrize("style", ["half", "interleaved"])
def test_rope_oracle_against_complex_turns_and_differences(style):
    r = np.random.default_rng(1)
    t, heads, hd, rot = 5, 2, 12, 8
    x, dy, g = r.standard_normal((t, heads, hd)), r.standard_normal((t, heads, hd)), r.standard_normal(hd)
    ang = r.uniform(0, 6, (20, rot // 2))
    cos, sin = np.cos(ang), np.sin(ang)
    pos = np.array([0, 7, -1, 19, 3])
    y = oqr.forward(x, g, 0.01, cos, sin, pos, style)
    u = x / np.sqrt((x ** 2).mean(-1, keepdims=True) + 0.01) * g
    a, b = (u[..., :rot // 2], u[..., rot // 2:rot]) if style == "half" else (u[..., 0:rot:2], u[..., 1:rot:2])
    z = (a + 1j * b) * np.exp(1j * ang[pos])[:, None]
    ya, yb = (y[..., :rot // 2], y[..., rot // 2:rot]) if style == "half" else (y[..., 0:rot:2], y[..., 1:rot:2])
    live = pos >= 0
    assert np.abs(ya - z.real)[live].max() < 1e-14 and np.abs(yb - z.imag)[live].max() < 1e-14
    assert np.abs(y - u)[live][..., rot:].max() < 1e-14 and not y[~live].any()
    dx, dg = oqr.backward(x, g, 0.01, cos, sin, pos, style, dy)
    for direction, of in ((r.standard_normal(x.shape), "x"), (r.standard_normal(hd), "g")):
        ends = []
        for h in (1e-6, -1e-6):
            args = (x + h * direction, g) if of == "x" else (x, g + h * direction)
            ends.append((oqr.forward(*args, 0.01, cos, sin, pos, style) * dy).sum())
        slope = (ends[0] - ends[1]) / 2e-6
        assert abs(((dx if of == "x" else dg) * direction).sum() - slope) < 1e-7
