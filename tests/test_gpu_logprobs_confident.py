"""Gradients of confident positions at large widths, row by row against 64 bits: there g (1 - p) of a confident token,
g - p sum g of a student that has met its teacher, and ln p + H of a low entropy are small differences of large
numbers, and an error that is small beside a probability is not small beside them.

Tolerances, derived before the first run. dz: the error of one logit, 2^-14 sum |e c| (test_gpu_logprobs). With errors
dy_v of the logits, |dy| <= dz / T, p_v is off by p_v (dy_v - sum_u p_u dy_u), at most 2 p_v (1 - p_v) dz / T, ln p_v by
2 (1 - p_v) dz / T, and H by sum_u p_u |ln p_u + H| dz / T: all vanish as a row grows confident, as long as the
backward's probabilities come from the logits that the statistics were formed of. What does not vanish is fp32 itself:
the sum S, between 1 and 2 there, is added up in fewer than 32 steps of 2^-24 each, so p_v is off by 2^-19 p_v, ln p_v
and H by 2^-18 (1 + |.|) with their own roundings. G is rounded to bf16 (2^-8 |G|; dC: its rows of E too), sums lose
2^-12 of the sum of magnitudes.
"""
import math

import pytest
import torch

from linear_cross_entropy_06_b200 import logprobs as L
from linear_cross_entropy_06_b200 import ops

from test_gpu_logprobs import logit_tol, reference

pytestmark = pytest.mark.gpu

V = 5000


def confident(N, D, seed, device):
    """Rows whose best token has 1 - p of about 0.1, 1e-3, 1e-4, 1e-5 in turn."""
    g = torch.Generator().manual_seed(seed)
    C = (torch.randn(V, D, generator=g) / math.sqrt(D)).bfloat16()
    best = torch.randint(0, V, (N,), generator=g)
    rest = torch.tensor([0.1, 1e-3, 1e-4, 1e-5])[torch.arange(N) % 4]
    c = C[best].double()
    alpha = (math.log(V) + 0.03 - rest.log().double()) / (c * c).sum(1)
    E = (0.25 * torch.randn(N, D, generator=g) + alpha[:, None] * c).bfloat16()
    return E.to(device), C.to(device), best.to(device), g


def tight_reference(E, C, tok, T, g, h):
    lp, H, p, logp, wanted = reference(E, C, None, tok, T)
    gw = torch.where(wanted, g.double(), 0.0)
    hw = torch.where(wanted.any(1), h.double(), 0.0)[:, None]
    total = gw.sum(1, keepdim=True)
    inner = logp + H[:, None]
    G = (-p * (total + hw * inner)).scatter_add_(1, tok.clamp(min=0), gw) / T
    dy = (logit_tol(E, C) / T)[:, None]
    rest = -torch.expm1(logp)
    dp = 2 * p * rest * dy + 2.0 ** -19 * p
    dlnp = 2 * rest * dy + 2.0 ** -18 * (1 + logp.abs())
    dH = (p * inner.abs()).sum(1, keepdim=True) * dy + 2.0 ** -18 * (1 + H[:, None])
    eG = (dp * (total.abs() + hw.abs() * inner.abs()) + hw.abs() * p * (dlnp + dH)) / T
    eG.scatter_add_(1, tok.clamp(min=0), gw.abs() * 2.0 ** -21 / T)
    eG += 2.0 ** -8 * G.abs()
    a = G.abs() + eG
    E, C = E.double(), C.double()
    return (G @ C, G.T @ E), (eG @ C.abs() + 2.0 ** -12 * (a @ C.abs()),
                              eG.T @ E.abs() + (2.0 ** -8 + 2.0 ** -12) * (a.T @ E.abs()))


def check(got, ref, tol):
    for name, x, r, t in zip(("dE", "dC"), got, ref, tol):
        worst = ((x.double() - r).abs() / (t + 1e-30)).amax(1)
        assert (worst <= 1).all(), f"{name}: {worst.max().item():.1f} of the tolerance, row {worst.argmax().item()}"


@pytest.mark.parametrize("D", [520, 2048, 4096])
@pytest.mark.parametrize("T", [1.0, 0.25])
def test_gradients_of_confident_tokens(device, D, T):
    """Half of the rows are given their best token, the others any: the best one's entry is then a probability only."""
    N = 160
    E, C, best, gen = confident(N, D, D, device)
    E = (E.double() * T).bfloat16()  # the same confidence at the temperature
    tok = torch.where(torch.arange(N, device=device) % 8 < 4, best, torch.randint(0, V, (N,), generator=gen).to(device))
    tok = tok[:, None]
    g, h = torch.randn(N, 1, generator=gen).to(device), torch.randn(N, generator=gen).to(device)
    lp, H, lse, *_ = L.cce_logprobs(E, C, tok, temperature=T, check=True)
    for gg, hh in ((g, h), (g, None), (None, h)):
        out = L.cce_logprobs_backward(E, C, tok, lp, lse, H, None, gg, hh, temperature=T, out_fp32=ops.OUT_FP32,
                                      check=True)
        check(out, *tight_reference(E, C, tok, T, torch.zeros_like(g) if gg is None else gg,
                                    torch.zeros_like(h) if hh is None else hh))


@pytest.mark.parametrize("D", [520, 4096])
def test_gradients_of_a_student_that_has_met_its_teacher(device, D):
    """Three tokens a row weighed by a teacher's probabilities that differ from the student's by a thousandth: every
    entry g - p sum g is a thousandth of its parts. One row gives a token twice."""
    N = 100
    E, C, best, gen = confident(N, D, 7 * D, device)
    tok = torch.randint(0, V, (N, 3), generator=gen).to(device)
    tok[:, 1] = best
    tok[5, 2] = tok[5, 1]
    _, _, p, _, _ = reference(E, C, None, tok, 1.0)
    noise = torch.randn(N, 3, generator=gen, dtype=torch.float64).to(device)
    share = p.gather(1, tok)
    g = (share / share.sum(1, keepdim=True) * (1 + 1e-3 * noise)).float()
    lp, H, lse, *_ = L.cce_logprobs(E, C, tok, check=True)
    out = L.cce_logprobs_backward(E, C, tok, lp, lse, H, None, g, None, out_fp32=ops.OUT_FP32, check=True)
    check(out, *tight_reference(E, C, tok, 1.0, g, torch.zeros(N, device=device)))
