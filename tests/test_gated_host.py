"""The gated feed-forward block without a GPU: its oracle against autograd, differences and an explicitly sharded form, and
the refusals of its calls, which come before anything reaches a device."""
import ctypes

import numpy as np
import pytest
import torch

import tensor_transformer_mlp_gb300 as tp
from oracle import gated as og
from tensor_transformer_mlp_gb300 import _binding

OK, INVALID, SHAPE, DTYPE, ALIGN, CUDA, TIMEOUT, WORKSPACE = range(8)
F32, BF16 = 0, 1
ACTS = ["silu", "gelu_tanh", "gelu_erf"]


def _inputs(n, d, m, seed=0):
    r = np.random.default_rng(seed)
    return r.standard_normal((n, d)), r.standard_normal((d, 2 * m)), r.standard_normal((m, d)), r.standard_normal((n, d))


def _torch_act(z, kind):
    if kind == "silu":
        return torch.nn.functional.silu(z)
    return torch.nn.functional.gelu(z, approximate="tanh" if kind == "gelu_tanh" else "none")


@pytest.mark.parametrize("kind", ACTS)
@pytest.mark.parametrize("t", [1, 3])
def test_oracle_against_autograd_over_shards(kind, t):
    n, d, m = 7, 10, 24
    X, A, B, G = _inputs(n, d, m)
    f = og.forward(X, A, B, t, kind)
    g = og.backward(X, A, B, G, f["Z"], f["Y"], t, kind)
    x, a, b = (torch.tensor(v, requires_grad=True) for v in (X, A, B))
    mt, o = m // t, 0
    for i in range(t):                     # a rank's slice of A is one [gate | up] matrix
        ai, bi = a[:, 2 * i * mt:2 * (i + 1) * mt], b[i * mt:(i + 1) * mt]
        z = x @ ai
        o = o + (_torch_act(z[:, :mt], kind) * z[:, mt:]) @ bi
    o.backward(torch.tensor(G))
    assert np.allclose(f["O"], o.detach().numpy(), rtol=1e-12, atol=1e-12)
    for k, v in (("dX", x), ("dA", a), ("dB", b)):
        assert np.allclose(g[k], v.grad.numpy(), rtol=1e-10, atol=1e-11), k


@pytest.mark.parametrize("kind", ACTS)
def test_oracle_gradients_against_differences(kind):
    n, d, m, t, step = 3, 4, 6, 2, 1e-6
    X, A, B, G = _inputs(n, d, m, seed=1)
    f = og.forward(X, A, B, t, kind)
    g = og.backward(X, A, B, G, f["Z"], f["Y"], t, kind)
    for k, v in (("dX", X), ("dA", A), ("dB", B)):
        for at in np.ndindex(v.shape):
            old = v[at]
            v[at] = old + step
            hi = (G * og.forward(X, A, B, t, kind)["O"]).sum()
            v[at] = old - step
            lo = (G * og.forward(X, A, B, t, kind)["O"]).sum()
            v[at] = old
            assert abs((hi - lo) / (2 * step) - g[k][at]) < 1e-6 * (1 + abs(g[k][at]))


# ----------------------------------------------------------------------- refusals

AT = [n << 40 for n in range(1, 16)]       # never dereferenced: every call fails validation first


@pytest.fixture(scope="module")
def lib():
    return _binding.load_library()


def fwd(lib, X=AT[0], A=AT[1], B=AT[2], O=AT[3], Z=AT[4], Y=AT[5], n=256, d=512, m=1024, t=2, act=2, dt=BF16, ws=AT[6],
        ws_bytes=1 << 30):
    return lib.tpmlp_gated_forward(X, A, B, O, Z, Y, n, d, m, t, act, dt, ws, ws_bytes, None)


def bwd(lib, X=AT[0], A=AT[1], B=AT[2], G=AT[3], Z=AT[4], Y=AT[5], dX=AT[6], dA=AT[7], dB=AT[8], n=256, d=512, m=1024, t=2,
        act=2, wgrad=0, dt=BF16, ws=AT[9], ws_bytes=None):
    if ws_bytes is None:
        ws_bytes = lib.tpmlp_gated_backward_workspace_size(n, d, m, dt)
    return lib.tpmlp_gated_backward(X, A, B, G, Z, Y, dX, dA, dB, n, d, m, t, act, wgrad, dt, ws, ws_bytes, None)


@pytest.mark.parametrize("call", [fwd, bwd])
def test_refusals(lib, call):
    assert call(lib, dt=F32) == DTYPE and b"bf16" in lib.tpmlp_last_error()
    assert call(lib, act=3) == INVALID and call(lib, act=-1) == INVALID
    assert call(lib, n=-1) == SHAPE and call(lib, d=0) == SHAPE and call(lib, m=0) == SHAPE
    assert call(lib, t=0) == SHAPE and call(lib, t=3) == SHAPE and b"divisible" in lib.tpmlp_last_error()
    assert call(lib, d=500) == SHAPE
    assert call(lib, m=8, t=2) == SHAPE            # shards of 4 columns
    assert call(lib, m=1 << 30, t=1) == SHAPE and call(lib, n=(1 << 31) - 1) == SHAPE
    for name in ("X", "A", "B", "Y"):
        assert call(lib, **{name: None}) == INVALID, name
        assert call(lib, **{name: AT[10] + 8}) == ALIGN, name
    assert call(lib, Z=AT[10] + 8) == ALIGN


def test_forward_refuses_overlaps(lib):
    assert fwd(lib, O=AT[0]) == INVALID and b"overlaps" in lib.tpmlp_last_error()
    assert fwd(lib, Z=AT[0] + 16) == INVALID
    assert fwd(lib, Y=AT[4] + 16) == INVALID                                  # across Z
    assert fwd(lib, Y=AT[1] + 512 * 2048 * 2 - 16) == INVALID                 # A's last columns
    assert fwd(lib, O=AT[2] - 16) == INVALID                                  # B's first


def test_backward_refusals_of_its_own(lib):
    assert bwd(lib, wgrad=3) == INVALID and bwd(lib, wgrad=-1) == INVALID
    for name in ("G", "Z", "dX", "dA", "dB"):
        assert bwd(lib, **{name: None}) == INVALID, name
    need = lib.tpmlp_gated_backward_workspace_size(256, 512, 1024, BF16)
    assert need >= 256 * 2048 * 2
    assert bwd(lib, ws_bytes=need - 1) == WORKSPACE and bwd(lib, ws=None) == WORKSPACE
    assert bwd(lib, ws=AT[9] + 16) == ALIGN
    assert bwd(lib, dX=AT[0]) == INVALID and bwd(lib, dA=AT[8]) == INVALID
    assert bwd(lib, dB=AT[9] + 256) == INVALID                                # the workspace
    # fp32 gradients take twice the bytes of bf16 ones: dB right behind bf16 dA meets fp32 dA
    assert bwd(lib, dB=AT[7] + 512 * 2048 * 2, wgrad=0) == INVALID


def test_no_tokens(lib):
    # nothing is launched: the token buffers may be null, the weights must be there
    assert fwd(lib, n=0, X=None, O=None, Z=None, Y=None, ws=None, ws_bytes=0) == OK
    assert fwd(lib, n=0, A=None) == INVALID
    assert bwd(lib, n=0, X=None, G=None, Z=None, Y=None, dX=None, ws=None, ws_bytes=0, wgrad=1) == OK
    assert lib.tpmlp_gated_backward_workspace_size(0, 64, 64, BF16) == 0
    assert lib.tpmlp_gated_forward_workspace_size(0, 64, 64, 1, BF16) == 0


def test_python_refusals():
    X, A, B = (torch.zeros(*s, dtype=torch.bfloat16) for s in ((4, 16), (16, 32), (16, 16)))
    with pytest.raises(ValueError, match="CUDA"):
        tp.gated_forward(X, A, B)
    with pytest.raises(ValueError, match="A must be"):
        tp.gated_forward(X, A[:, :16].contiguous(), B)
    with pytest.raises(ValueError, match="X must be"):
        tp.gated_forward(X.T.contiguous().T, A, B)
    G, Z, Y = torch.zeros_like(X), torch.zeros(4, 32, dtype=X.dtype), torch.zeros(4, 16, dtype=X.dtype)
    with pytest.raises(ValueError, match="f32_add"):
        tp.gated_backward(X, A, B, G, Z, Y, wgrad="f32_add")
    with pytest.raises(ValueError, match="dA must be"):
        tp.gated_backward(X, A, B, G, Z, Y, wgrad="operand", dA=torch.zeros(16, 32))
    with pytest.raises(ValueError, match="Z must be"):
        tp.gated_backward(X, A, B, G, Z[:, :16].contiguous(), Y)
    with pytest.raises(KeyError):
        tp.gated_backward(X.float(), A.float(), B.float(), G.float(), Z.float(), Y.float(), wgrad="f64", dA=None)
