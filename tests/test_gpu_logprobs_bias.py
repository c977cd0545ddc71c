"""The gradient of a bias comes in the bias's own type: in fp32 it is not rounded to bf16 on the way.

Tolerance: as in test_gpu_logprobs, without the rounding of G and of the output to bf16 (the column sums are those of G
in fp32): the error of p, 2^-22 of a token's own gradient, 2^-12 of the sum of magnitudes."""
import pytest
import torch

import linear_cross_entropy_06_b200 as lce

from test_gpu_logprobs import logit_tol, make, reference

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.float32, torch.float64, torch.bfloat16])
@pytest.mark.parametrize("eps", [0.0, 2.0 ** -30])
def test_gradient_of_the_bias_in_its_own_type(device, dtype, eps):
    N, D, V, K, T = 60, 128, 3000, 3, 0.8
    E, C, bias, tok = make(N, D, V, 1, device, True, K)
    gen = torch.Generator().manual_seed(2)
    g, h = torch.randn(N, K, generator=gen).to(device), torch.randn(N, generator=gen).to(device)
    b = bias.to(dtype).requires_grad_(True)
    out = lce.linear_logprobs(E, C, tok, bias=b, temperature=T, filter_eps=eps)
    (got,) = torch.autograd.grad((out.logprobs, out.entropy), b, (g, h))
    assert got.dtype == dtype
    _, H, p, logp, wanted = reference(E, C, bias, tok, T)
    gw = torch.where(wanted, g.double(), 0.0)
    hw = torch.where(wanted.any(1), h.double(), 0.0)[:, None]
    total, inner = gw.sum(1, keepdim=True), logp + H[:, None]
    G = (-p * (total + hw * inner)).scatter_add_(1, tok.clamp(min=0), gw) / T
    dz = (2 * logit_tol(E, C) / T + 2.0 ** -18)[:, None]
    mag = p * (total.abs() + hw.abs() * (logp.abs() + H[:, None])) / T
    eG = mag * (dz + 2.0 ** -20) + p * hw.abs() * dz / T
    eG.scatter_add_(1, tok.clamp(min=0), gw.abs() / T * 2.0 ** -22)
    want = G.sum(0)
    tol = eG.sum(0) + 2.0 ** -12 * (G.abs() + eG).sum(0) + 1e-30
    if eps > 0:
        tol += N * 2.0 ** -30 * (total.abs().amax() + hw.abs().amax() * 30) / T
    if dtype == torch.bfloat16:
        tol += 2.0 ** -8 * (want.abs() + tol)
    worst = ((got.double() - want).abs() / tol).max().item()
    assert worst <= 1, f"{worst:.1f} of the tolerance"


def test_no_rows(device):
    E, C, bias, _ = make(4, 64, 300, 3, device, True)
    b = bias.float().requires_grad_(True)
    out = lce.linear_logprobs(E[:0], C, torch.zeros(0, dtype=torch.int64, device=device), bias=b)
    (got,) = torch.autograd.grad(out.logprobs.sum() + out.entropy.sum(), b)
    assert got.dtype == torch.float32 and got.shape == (300,) and (got == 0).all()
