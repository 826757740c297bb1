"""The norms around a block where a value that the formula does not read is infinite or NaN."""
import pytest
import torch

import tensor_transformer_mlp_gb300 as tp

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


# (b, s, h, type): rows of lane groups, of a warp, and of a CTA, from a ring, held in registers and read where they lie
@pytest.mark.parametrize("b,s,h,dtype", [(2, 40, 64, BF16), (2, 40, 320, F32), (2, 2500, 320, BF16), (2, 2500, 512, F32),
                                         (2, 2500, 1000, BF16), (2, 40, 776, BF16), (2, 40, 2048, BF16), (2, 40, 4096, BF16),
                                         (2, 40, 8192, BF16), (2, 40, 1608, F32), (2, 40, 4096, F32), (2, 40, 5000, F32)])
@pytest.mark.parametrize("pre", [False, True])
def test_gradients_of_an_unnormed_block_output_do_not_read_it(b, s, h, dtype, pre):
    # without gamma_post, dy = gate g: y is in dgate alone
    gen = torch.Generator("cuda").manual_seed(h)
    y, r, dr, du = (torch.randn(b, s, h, generator=gen, device="cuda").to(dtype) for _ in range(4))
    gains = dict(gate=torch.randn(b, h, generator=gen, device="cuda"))
    if pre:
        gains["gamma_pre"] = 1 + 0.1 * torch.randn(h, generator=gen, device="cuda")
    else:
        du = None
    want = tp.residual_norm_backward(y, r, dr, du, **gains)
    bad = y.clone()
    bad[0, 3, 5], bad[0, 9, 6], bad[1, 7, 2] = float("inf"), -float("inf"), float("nan")
    bad[1, 8, 8:] = float("inf")
    got = tp.residual_norm_backward(bad, r, dr, du, **gains)
    torch.cuda.synchronize()
    tp.tpmlp_device_status()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    ok = torch.ones(b, h, dtype=torch.bool, device="cuda")
    ok[0, 5:7] = ok[1, 2] = False
    ok[1, 8:] = False
    assert torch.equal(got[3][ok], want[3][ok]) and not torch.isfinite(got[3][~ok]).any()
    if pre:
        assert torch.equal(got[4], want[4])
