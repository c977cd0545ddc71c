"""Gradients at small temperatures, where lse = z_max / T + ln S is so large (4e6 here) that its fp32 step is more than
the probabilities bear, on logits that every order of summation forms exactly.

Logits are base + j 2^-18 with bases of 8 to 12 in steps of 1/16 and whole j: 22 bits, so neither the tensor cores nor
fp32 lose any, and only the probabilities' own roundings are left. Tolerances, derived before the first run: z - z_max is
exact, its product with log2(e) / T carries four roundings of 2^-24 (ln p to 2^-22 |ln p|), ln S, its product with
log2(e) and the sum S another 2^-20 each at S < 300, the exponential 2^-22: ln p and p are within 2^-18 (1 + |ln p|), H
within 2^-18 (1 + H) more. G is rounded to bf16 (2^-8), for dC its rows of E too, sums lose 2^-12 of the sum of
magnitudes, outputs are rounded to bf16.
"""
import ctypes

import pytest
import torch

import linear_cross_entropy_06_b200 as lce

pytestmark = pytest.mark.gpu

N, D, V = 150, 64, 300


def exact_logits(device, seed):
    g = torch.Generator().manual_seed(seed)
    E, C = torch.zeros(N, D), torch.zeros(V, D)
    E[:, 0] = 8 + torch.randint(0, 65, (N,), generator=g) / 16
    E[:, 1] = 1
    C[:, 0] = 1
    C[:, 1] = torch.randint(0, 100, (V,), generator=g) * 2.0 ** -18
    E[:, 2:] = torch.randint(-3, 4, (N, D - 2), generator=g)  # these meet zeros in C: they show in dC
    return E.bfloat16().to(device), C.bfloat16().to(device), g


@pytest.mark.parametrize("T", [1e-6, 2.0 ** -19, 1e-5, 1e-3])
@pytest.mark.parametrize("K", [1, 3])
def test_gradients_at_small_temperatures(device, T, K):
    E, C, g = exact_logits(device, K)
    z = E.double() @ C.double().T
    assert torch.equal(z.float().double(), z)
    tok = torch.randint(0, V, (N, K), generator=g).to(device)
    tok[::2, 0] = z[::2].argmax(1)
    gl, h = torch.randn(N, K, generator=g).to(device), torch.randn(N, generator=g).to(device)
    e, c = E.clone().requires_grad_(True), C.clone().requires_grad_(True)
    out = lce.linear_logprobs(e, c, tok, temperature=T)
    t = ctypes.c_float(T).value
    logp = torch.log_softmax(z / t, 1)
    p, H = logp.exp(), torch.special.entr(logp.exp()).sum(1)
    want = logp.gather(1, tok)
    assert ((out.logprobs.double() - want).abs() <= 2.0 ** -18 * (1 + want.abs())).all()
    assert ((out.entropy.double() - H).abs() <= 2.0 ** -18 * (1 + H)).all()
    for gg, hh in ((gl, h), (gl, torch.zeros_like(h)), (torch.zeros_like(gl), h)):
        got = torch.autograd.grad((out.logprobs, out.entropy), (e, c), (gg, hh), retain_graph=True)
        gw, hw = gg.double(), hh.double()[:, None]
        total, inner = gw.sum(1, keepdim=True), logp + H[:, None]
        G = (-p * (total + hw * inner)).scatter_add_(1, tok, gw) / t
        dlnp = 2.0 ** -18 * (1 + logp.abs())
        eG = p * (dlnp * (total.abs() + hw.abs() * inner.abs()) + hw.abs() * (dlnp + 2.0 ** -18 * (1 + H[:, None]))) / t
        # p below the smallest normal number of fp32 counts as 0 (ln p = -89.5 at 8.8e-5 below the largest logit and
        # T = 1e-6: p = 1.3e-39, 2^-129), and 1 / T raises what is lost there to 1e-32
        eG += 2.0 ** -126 * (total.abs() + hw.abs() * inner.abs()) / t
        eG.scatter_add_(1, tok, gw.abs() * 2.0 ** -21 / t)
        eG += 2.0 ** -8 * G.abs()
        a = G.abs() + eG
        x, y = E.double(), C.double()
        refs = (G @ y, G.T @ x)
        tols = (eG @ y.abs() + 2.0 ** -12 * (a @ y.abs()), eG.T @ x.abs() + (2.0 ** -8 + 2.0 ** -12) * (a.T @ x.abs()))
        for name, have, r, tol in zip(("dE", "dC"), got, refs, tols):
            tol = tol + 1e-30 + 2.0 ** -8 * (r.abs() + tol)
            worst = ((have.double() - r).abs() / tol).max().item()
            assert worst <= 1, f"{name}: {worst:.1f} of the tolerance"


@pytest.mark.parametrize("fill", [torch.finfo(torch.bfloat16).min, torch.finfo(torch.bfloat16).max / 4])
def test_logits_whose_quotient_leaves_the_range_of_fp32(device, fill):
    """z / T is beyond fp32, and so is lse, but the probabilities are not: all logits are equal, p = 1 / V."""
    E, C, g = exact_logits(device, 5)
    bias = torch.full((V,), fill, dtype=torch.bfloat16, device=device)
    tok = torch.randint(0, V, (N, 2), generator=g).to(device)
    gl = torch.randn(N, 2, generator=g).to(device)
    T = 0.125
    e, c = E.clone().requires_grad_(True), C.clone().requires_grad_(True)
    out = lce.linear_logprobs(e, c, tok, bias=bias, temperature=T)
    ln_v = torch.tensor(float(V)).log()
    assert ((out.logprobs + ln_v).abs() <= 2.0 ** -18 * 7).all() and ((out.entropy - ln_v).abs() <= 2.0 ** -18 * 7).all()
    got = torch.autograd.grad((out.logprobs, out.entropy), (e, c), (gl, torch.zeros(N, device=device)))
    gw = gl.double()
    G = (-gw.sum(1, keepdim=True) / V).expand(N, V).clone().scatter_add_(1, tok, gw) / T
    x, y = E.double(), C.double()
    for have, r, mag, own in zip(got, (G @ y, G.T @ x), (G.abs() @ y.abs(), G.abs().T @ x.abs()), (2, 3)):
        tol = (own * 2.0 ** -8 + 2.0 ** -12) * mag  # G and the outputs rounded to bf16, for dC the rows of E too
        assert ((have.double() - r).abs() <= tol + 2.0 ** -8 * (r.abs() + tol)).all()
