"""Tensors of more than 2^31 values: the gated block's Z and the norms' rows, sampled where offsets pass 32 bits."""
import pytest
import torch

import tensor_transformer_mlp_gb300 as tp

pytestmark = pytest.mark.gpu


def test_gated_block_with_z_past_32_bits():
    # 70016 x 32768 values of Z, 4.6 GB. Sampled rows against 64 bits: half a step of bf16 for each rounding, two roundings in
    # O of which the inner ones add up like noise (2^-8 / sqrt(3), 7 deviations).
    n, d, m, t = 70016, 64, 16384, 4
    gen = torch.Generator("cuda").manual_seed(0)
    X, G = (torch.randn(n, d, generator=gen, device="cuda").bfloat16() for _ in range(2))
    A = (d ** -0.5 * torch.randn(d, 2 * m, generator=gen, device="cuda")).bfloat16()
    B = (m ** -0.5 * torch.randn(m, d, generator=gen, device="cuda")).bfloat16()
    O, Z, Y = tp.gated_forward(X, A, B, t)
    dX, dA, dB = tp.gated_backward(X, A, B, G, Z, Y, t)
    torch.cuda.synchronize()
    tp.tpmlp_device_status()
    rows = torch.tensor([0, 255, 256, 65535, 65536, 65537, n - 1], device="cuda")
    a, b = A.double(), B.double()
    z = X[rows].double() @ a
    assert ((Z[rows].double() - z).abs() <= 2.0 ** -8 * z.abs() + 1e-5).all()
    zz = Z[rows].double().requires_grad_()
    parts = zz.view(-1, t, 2, m // t)
    y = (torch.nn.functional.silu(parts[:, :, 0]) * parts[:, :, 1]).reshape(-1, m)
    noise = 2.0 ** -8 / 3 ** 0.5
    assert ((Y[rows].double() - y).norm() / y.norm()).item() <= 3 * noise      # its own rounding, and those of both parts of Z
    o = Y[rows].double() @ b
    assert ((O[rows].double() - o).abs() <= 2.0 ** -8 * o.abs() + 1e-5).all()
    dz, = torch.autograd.grad(y, zz, G[rows].double() @ b.T)
    want = dz @ a.T
    bound = 2.0 ** -8 * want.abs() + 7 * noise * ((dz * dz) @ (a * a).T).sqrt() + 1e-5
    assert ((dX[rows].double() - want).abs() <= bound).all()
    # all rows count in dB: its columns of the last shard against chunks in 64 bits, fp32 sums of n terms (n / 16 steps of 2^-22)
    cols = torch.arange(m - 8, m, device="cuda")
    ref, mag = torch.zeros(8, d, dtype=torch.float64, device="cuda"), torch.zeros(8, d, dtype=torch.float64, device="cuda")
    for k in range(0, n, 8192):
        yk, gk = Y[k:k + 8192, cols].double(), G[k:k + 8192].double()
        ref += yk.T @ gk
        mag += yk.abs().T @ gk.abs()
    assert ((dB[cols].double() - ref).abs() <= n / 16 * 2.0 ** -22 * mag).all()


def test_norms_with_rows_past_32_bits():
    # 540000 x 4096 values, 4.4 GB a tensor; the last rows, one CTA's neighbours and the first
    b, s, h = 3, 180000, 4096
    gen = torch.Generator("cuda").manual_seed(0)

    def draw():
        out = torch.empty(b, s, h, dtype=torch.bfloat16, device="cuda")
        for i in range(b):
            out[i] = torch.randn(s, h, generator=gen, device="cuda").bfloat16()
        return out
    x, y = draw(), draw()
    post, pre = (1 + 0.1 * torch.randn(h, generator=gen, device="cuda") for _ in range(2))
    gate = torch.randn(b, h, generator=gen, device="cuda")
    r, u = tp.residual_norm(x, y, post, gate, pre)
    dx, dy, dpost, dgate, dpre = tp.residual_norm_backward(y, r, x, u, post, gate, pre)   # any dr and du will do
    torch.cuda.synchronize()
    tp.tpmlp_device_status()
    at = [(0, 0), (1, 77), (2, 164288), (2, 164289), (2, s - 1)]

    def rms(v, g):
        return v / torch.sqrt((v * v).mean(-1, keepdim=True) + 1e-5) * g
    for i, j in at:
        X, Yv, R, DU = (v[i, j].double() for v in (x, y, r, u))
        want = X + gate[i].double() * rms(Yv, post.double())
        assert ((r[i, j].double() - want).abs() <= 2.0 ** -8 * want.abs() + 1e-5 * (1 + X.abs())).all()
        wu = rms(want, pre.double())
        assert ((u[i, j].double() - wu).abs() <= 2.0 ** -8 * wu.abs() + 1e-5 * (1 + wu.abs())).all()
        yy, rr = Yv.clone().requires_grad_(), R.clone().requires_grad_()
        g = X + torch.autograd.grad(rms(rr, pre.double()), rr, DU)[0]
        wy, = torch.autograd.grad(gate[i].double() * rms(yy, post.double()), yy, g)
        assert ((dx[i, j].double() - g).abs() <= 2.0 ** -8 * g.abs() + 1e-5 * (1 + g.abs())).all()
        assert ((dy[i, j].double() - wy).abs() <= 2.0 ** -8 * wy.abs() + 1e-5 * (1 + wy.abs())).all()
