"""Sums over tokens of tensors of more than 2^31 values: the gated block's dA, and the gains' and gates' gradients of the norms,
against chunks in 64 bits. Tolerances as in test_gpu_gated.py and test_gpu_residual_norm.py."""
import pytest
import torch

import tensor_transformer_mlp_gb300 as tp

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("wgrad", ["f32", "operand"])
def test_weight_gradient_of_a_d_past_32_bits(wgrad):
    # 70016 x 32768 values of D, read along its rows for dA: the first columns, and the last gate and up columns of the last shard
    n, d, m, t = 70016, 64, 16384, 4
    gen = torch.Generator("cuda").manual_seed(1)
    X, G = (torch.randn(n, d, generator=gen, device="cuda").bfloat16() for _ in range(2))
    A = (d ** -0.5 * torch.randn(d, 2 * m, generator=gen, device="cuda")).bfloat16()
    B = (m ** -0.5 * torch.randn(m, d, generator=gen, device="cuda")).bfloat16()
    _, Z, Y = tp.gated_forward(X, A, B, t)
    dA = tp.gated_backward(X, A, B, G, Z, Y, t, wgrad=wgrad)[1]
    torch.cuda.synchronize()
    tp.tpmlp_device_status()
    mt = m // t
    for y0 in (0, m - 8):
        shard, j = y0 // mt, y0 % mt
        gate = torch.arange(2 * shard * mt + j, 2 * shard * mt + j + 8, device="cuda")
        cols = torch.cat([gate, gate + mt])
        ref, mag, var = (torch.zeros(d, 16, dtype=torch.float64, device="cuda") for _ in range(3))
        b = B[y0:y0 + 8].double()
        for k in range(0, n, 8192):
            x, g, z = X[k:k + 8192].double(), G[k:k + 8192].double(), Z[k:k + 8192, cols].double().requires_grad_()
            y = torch.nn.functional.silu(z[:, :8]) * z[:, 8:]
            D, = torch.autograd.grad(y, z, g @ b.T)
            ref += x.T @ D
            mag += x.abs().T @ D.abs()
            # D is rounded to bf16; its dY is a sum of d terms in fp32
            off = (d / 16 + 1) * 2.0 ** -22 * (g.abs() @ b.abs().T).repeat(1, 2) * (z.detach().abs().roll(8, 1) + 1) * 1.2
            var += (x * x).T @ ((2.0 ** -8 / 3 ** 0.5 * D) ** 2 + off ** 2)
        out = 2.0 ** -8 * ref.abs() if wgrad == "operand" else 2.0 ** -23 * ref.abs()
        assert ((dA[:, cols].double() - ref).abs() <= out + 7 * var.sqrt() + (n / 16 + 1) * 2.0 ** -22 * mag).all(), y0


def test_norms_sums_over_rows_past_32_bits():
    # 540000 x 4096 values: every sequence crosses CTAs, so each row of dgate is joined from them
    b, s, h, eps = 3, 180000, 4096, 1e-5
    gen = torch.Generator("cuda").manual_seed(2)

    def draw():
        out = torch.empty(b, s, h, dtype=torch.bfloat16, device="cuda")
        for i in range(b):
            out[i] = torch.randn(s, h, generator=gen, device="cuda").bfloat16()
        return out
    y, r, du = draw(), draw(), draw()
    dr = r.flip(1)
    post, pre = (1 + 0.1 * torch.randn(h, generator=gen, device="cuda") for _ in range(2))
    gate = torch.randn(b, h, generator=gen, device="cuda")
    dpost, dgate, dpre = tp.residual_norm_backward(y, r, dr, du, post, gate, pre, dx=torch.empty_like(y), dy=torch.empty_like(y))[2:]
    torch.cuda.synchronize()
    tp.tpmlp_device_status()
    cols = torch.tensor([0, 1, 1000, 2047, 2048, 4094, 4095], device="cuda")
    zeros = (torch.zeros(b, len(cols), dtype=torch.float64, device="cuda") for _ in range(4))
    S, S_mag, P, P_mag = zeros                             # sums of g y_hat and of du r_hat, and of their magnitudes
    w, p64 = pre.double(), post.double()
    for i in range(b):
        for k in range(0, s, 6000):
            Y, R, U, DR = (v[i, k:k + 6000].double() for v in (y, r, du, dr))
            ry, rr = (1 / torch.sqrt((v * v).mean(-1, keepdim=True) + eps) for v in (Y, R))
            c = (U * w * R * rr).mean(-1, keepdim=True)
            c_mag = (U * w * R * rr).abs().mean(-1, keepdim=True)
            Yc, Rc, Uc, Dc = (v[:, cols] for v in (Y, R, U, DR))
            g = Dc + rr * (Uc * w[cols] - Rc * rr * c)
            g_mag = Dc.abs() + rr * ((Uc * w[cols]).abs() + (Rc * rr).abs() * c_mag)
            S[i] += (g * Yc * ry).sum(0)
            S_mag[i] += (g_mag * (Yc * ry).abs()).sum(0)
            P[i] += (Uc * Rc * rr).sum(0)
            P_mag[i] += (Uc * Rc * rr).abs().sum(0)
    many = 8 * (b * s) ** 0.5 * 2.0 ** -24 + 2.0 ** -18
    gc = gate[:, cols].double()
    assert ((dgate[:, cols].double() - p64[cols] * S).abs() <= many * p64[cols].abs() * S_mag).all()
    assert ((dpost[cols].double() - (gc * S).sum(0)).abs() <= many * (gc.abs() * S_mag).sum(0)).all()
    assert ((dpre[cols].double() - P.sum(0)).abs() <= many * P_mag.sum(0)).all()
