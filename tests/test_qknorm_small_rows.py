"""The norm's gradient of rows near float32's smallest normal sizes, with eps = 0: 1 / rms is about 2^61.

Tolerance: that of the other gradients, 2^-18 of the sizes that cancel, and the outputs' rounding."""
import pytest
import torch

import _attn_ref as ref

pytestmark = pytest.mark.gpu
F64 = torch.float64


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("d", [64, 128, 30])
def test_gradient_of_small_rows(kda, d, inter, dtype):
    g = torch.Generator().manual_seed(1)
    x = (torch.randn(50, 3, d, generator=g) * 3e-19).to(dtype)
    dy = (torch.randn(50, 3, d, generator=g) * 1000).to(dtype)
    w = 1 + 0.1 * torch.randn(d, generator=g)
    pos = torch.arange(50, dtype=torch.int32)
    freqs = 0.5 ** torch.arange(d // 2 if d > 30 else 8, dtype=F64)
    dx, _, dw, _ = kda.qknorm_bwd(x.cuda(), None, dy.cuda(), None, pos.cuda(), freqs.cuda(), q_weight=w.cuda(), interleaved=inter,
                                  eps=0.0)
    xd, wd = x.to(F64).requires_grad_(), w.to(F64).requires_grad_()
    gx, gw = torch.autograd.grad((ref.qknorm(xd, pos, freqs, wd, inter, eps=0.0) * dy.to(F64)).sum(), (xd, wd))
    size = (dy.to(F64).abs().amax(-1, keepdim=True) * 2) * torch.rsqrt(x.to(F64).square().mean(-1, keepdim=True)) \
        + gx.abs().amax(-1, keepdim=True)
    half = 2.0 ** -24 if dtype is torch.float32 else 2.0 ** -8
    assert ((dx.cpu().to(F64) - gx).abs() <= gx.abs() * half + 2.0 ** -18 * size).all()
    assert ((dw.cpu().to(F64) - gw).abs() <= 2.0 ** -18 * 150 * 4000 * 4).all()
