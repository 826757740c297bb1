"""The norms around a block without a GPU: their oracle against autograd and differences, and the refusals of the calls."""
import itertools

import numpy as np
import pytest
import torch

import tensor_transformer_mlp_gb300 as tp
from oracle import residual_norm as orn
from tensor_transformer_mlp_gb300 import _binding

OK, INVALID, SHAPE, DTYPE, ALIGN, CUDA, TIMEOUT, WORKSPACE = range(8)
F32, BF16 = 0, 1
FORMS = list(itertools.product([False, True], repeat=3))   # post, gate, pre


def _case(form, b=2, s=3, h=8, seed=0):
    g = np.random.default_rng(seed)
    x, y, dr, du = (g.standard_normal((b, s, h)) for _ in range(4))
    post, pre = (g.standard_normal(h) if on else None for on in (form[0], form[2]))
    gate = g.standard_normal((b, h)) if form[1] else None
    return x, y, dr, du if form[2] else None, post, gate, pre


@pytest.mark.parametrize("form", FORMS)
def test_oracle_against_autograd(form):
    x, y, dr, du, post, gate, pre = _case(form)
    alpha, eps = 0.7, 1e-3
    t = {k: torch.tensor(v, requires_grad=True) for k, v in dict(x=x, y=y, post=post, gate=gate, pre=pre).items() if v is not None}
    p = t["y"]
    if form[0]:
        p = torch.nn.functional.rms_norm(p, (8,), t["post"], eps)
    if form[1]:
        p = p * t["gate"][:, None]
    r = alpha * t["x"] + p
    loss = (r * torch.tensor(dr)).sum()
    rn, un = orn.forward(x, y, post, gate, pre, alpha, eps)
    assert np.allclose(rn, r.detach().numpy(), rtol=1e-12)
    if form[2]:
        u = torch.nn.functional.rms_norm(r, (8,), t["pre"], eps)
        loss = loss + (u * torch.tensor(du)).sum()
        assert np.allclose(un, u.detach().numpy(), rtol=1e-12)
    loss.backward()
    got = orn.backward(y, rn, dr, du, post, gate, pre, alpha, eps)
    assert set(got) == {"d" + k for k in t}
    for k, v in t.items():
        assert np.allclose(got["d" + k], v.grad.numpy(), rtol=1e-9, atol=1e-11), k


def test_oracle_gradients_against_differences():
    x, y, dr, du, post, gate, pre = _case((True, True, True), seed=1)
    alpha, eps, step = 1.3, 1e-3, 1e-6
    r, _ = orn.forward(x, y, post, gate, pre, alpha, eps)
    got = orn.backward(y, r, dr, du, post, gate, pre, alpha, eps)

    def loss():
        r, u = orn.forward(x, y, post, gate, pre, alpha, eps)
        return (r * dr).sum() + (u * du).sum()
    for k, v in (("dx", x), ("dy", y), ("dpost", post), ("dgate", gate), ("dpre", pre)):
        for at in np.ndindex(v.shape):
            old = v[at]
            v[at] = old + step
            hi = loss()
            v[at] = old - step
            lo = loss()
            v[at] = old
            assert abs((hi - lo) / (2 * step) - got[k][at]) < 1e-6 * (1 + abs(got[k][at])), k


# ----------------------------------------------------------------------- refusals

AT = [n << 40 for n in range(1, 20)]       # never dereferenced: every call fails validation first


@pytest.fixture(scope="module")
def lib():
    return _binding.load_library()


def fwd(lib, x=AT[0], y=AT[1], post=AT[2], gate=AT[3], pre=AT[4], alpha=1.0, eps=1e-5, r=AT[5], u=AT[6], b=2, s=16, h=64,
        dt=BF16):
    return lib.tpmlp_residual_norm(x, y, post, gate, pre, alpha, eps, r, u, b, s, h, dt, None)


def bwd(lib, y=AT[0], r=AT[1], dr=AT[2], du=AT[3], post=AT[4], gate=AT[5], pre=AT[6], alpha=1.0, eps=1e-5, dx=AT[7], dy=AT[8],
        dpost=AT[9], dgate=AT[10], dpre=AT[11], b=2, s=16, h=64, dt=BF16, ws=AT[12], ws_bytes=1 << 30):
    return lib.tpmlp_residual_norm_backward(y, r, dr, du, post, gate, pre, alpha, eps, dx, dy, dpost, dgate, dpre, b, s, h, dt,
                                            ws, ws_bytes, None)


@pytest.mark.parametrize("call", [fwd, bwd])
def test_refusals(lib, call):
    assert call(lib, dt=2) == DTYPE
    assert call(lib, b=-1) == SHAPE and call(lib, s=-1) == SHAPE and call(lib, b=1 << 20, s=1 << 20) == SHAPE
    assert call(lib, h=0) == SHAPE and call(lib, h=12) == SHAPE and call(lib, h=8200) == SHAPE
    assert call(lib, eps=0.0) == INVALID and call(lib, eps=float("nan")) == INVALID and call(lib, eps=float("inf")) == INVALID
    assert call(lib, alpha=float("inf")) == INVALID
    assert call(lib, y=None) == INVALID and call(lib, y=AT[13] + 8) == ALIGN
    for name in ("post", "gate", "pre"):
        assert call(lib, **{name: AT[13] + 8}) == ALIGN, name


def test_forward_refusals_of_its_own(lib):
    assert fwd(lib, x=None) == INVALID and fwd(lib, r=None) == INVALID
    assert fwd(lib, pre=None) == INVALID and fwd(lib, u=None) == INVALID and b"go together" in lib.tpmlp_last_error()
    assert fwd(lib, r=AT[6]) == INVALID                                     # r and u the same
    assert fwd(lib, r=AT[0] + 16) == INVALID and fwd(lib, u=AT[1] - 16) == INVALID
    assert fwd(lib, r=AT[2]) == INVALID and fwd(lib, u=AT[3] + 64 * 4) == INVALID   # gamma_post; the gate's second row
    assert fwd(lib, u=AT[6] + 4) == ALIGN


def test_backward_refusals_of_its_own(lib):
    for name in ("dpost", "dgate", "dpre"):
        assert bwd(lib, **{name: None}) == INVALID and b"go with" in lib.tpmlp_last_error()
        assert bwd(lib, **{name: AT[13] + 4}) == ALIGN
        assert bwd(lib, **{name: AT[0]}) == INVALID                         # y
    assert bwd(lib, du=None) == INVALID and bwd(lib, r=None) == INVALID
    assert bwd(lib, pre=None, dpre=None) == INVALID                         # du without gamma_pre
    assert bwd(lib, dr=None, du=None, pre=None, dpre=None) == INVALID
    assert bwd(lib, dx=None) == INVALID and bwd(lib, dy=None) == INVALID and bwd(lib, dx=AT[8]) == INVALID
    assert bwd(lib, dx=AT[2] + 16) == INVALID and bwd(lib, dy=AT[0] - 16) == INVALID
    need = lib.tpmlp_residual_norm_backward_workspace_size(2, 16, 64, 1)
    assert need >= 4 * 32 * 64 * 4
    assert need > lib.tpmlp_residual_norm_backward_workspace_size(2, 16, 64, 0)
    assert bwd(lib, ws_bytes=need - 1) == WORKSPACE and bwd(lib, ws=None) == WORKSPACE
    assert bwd(lib, ws=AT[12] + 128) == ALIGN and bwd(lib, ws=AT[5]) == INVALID


def test_no_tokens(lib):
    assert fwd(lib, b=0, x=None, y=None, r=None) == OK and fwd(lib, s=0) == OK
    assert lib.tpmlp_residual_norm_backward_workspace_size(0, 4, 64, 1) == 0
    assert bwd(lib, b=0, post=None, gate=None, pre=None, dpost=None, dgate=None, dpre=None, ws=None, ws_bytes=0) == OK


def test_python_refusals():
    x = torch.zeros(2, 3, 16)
    g, gate = torch.ones(16), torch.ones(2, 16)
    with pytest.raises(ValueError, match="CUDA"):
        tp.residual_norm(x, x, g, gate, g)
    with pytest.raises(ValueError, match="x must be"):
        tp.residual_norm(x.bfloat16(), x, g)
    with pytest.raises(ValueError, match="gate must be"):
        tp.residual_norm(x, x, g, torch.ones(3, 16))
    with pytest.raises(ValueError, match=r"\[b, h\]"):
        tp.residual_norm(x.view(6, 16), x.view(6, 16), g, gate)
    with pytest.raises(ValueError, match="u needs"):
        tp.residual_norm(x, x, g, u=x)
    with pytest.raises(ValueError, match="gamma_pre must be"):
        tp.residual_norm(x, x, g, gate, g.double())
    with pytest.raises(ValueError, match="dr must be"):
        tp.residual_norm_backward(x, x, x[:, :2].contiguous(), x, g, gate, g)
