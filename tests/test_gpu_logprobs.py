"""Log-probabilities of given tokens, entropy, top alternatives and 8-bit logits on the GPU, against the
definitions in 64 bits (plain torch on the same inputs).

Tolerances, derived before the first run. u = 2^-24 is half a step of fp32, 2^-8 that of bf16.
 logits   the tensor cores add 16 products and the running sum a step, each cut at 2^-24 of the largest (not
          rounded): at most 17 * 2^-24 * A a step, A = sum_d |e_d c_d|. A part of 512 values takes 32 steps, the
          parts' partial magnitudes add up to A, and their sums are rounded to nearest (under 2^-20 A):
          dz <= 32 * 17 * 2^-24 A + 2^-20 A < 2^-14 A.
 logprob  two logits (the token's, and a mean of them in lse), and fp32 roundings of the statistics: V terms
          summed in blocks of 64, each term a few u: 2 dz / T + 2^-18 (1 + |lp|).
 entropy  dH = -sum_v p_v (ln p_v + H) dy_v, and sum p |ln p + H| <= 2 H: 2 H dz / T + 2^-18 (1 + H).
 grads    G = p (coef + coef_log ln p) + onehot terms, relative error of p 2 dz / T (2^-18 more for its own
          roundings), one rounding to bf16 (2^-8 |G|), for dC one of the scaled rows of E (2^-8 |G| |E|), fp32 sums
          (2^-12 of the sum of magnitudes, with the cut sums of the tensor cores), and for bf16 outputs one more
          rounding.
"""
import math

import pytest
import torch

import linear_cross_entropy_06_b200 as lce
from linear_cross_entropy_06_b200 import logprobs as L
from linear_cross_entropy_06_b200 import ops

pytestmark = pytest.mark.gpu

IGNORE = -100


def make(N, D, V, seed, device, bias=False, K=None, alpha=6.0, ignore=0.1):
    g = torch.Generator(device="cpu").manual_seed(seed)
    C = torch.randn(V, D, generator=g) / math.sqrt(D)
    best = torch.randint(0, V, (N,), generator=g)
    E = (torch.randn(N, D, generator=g) + alpha * C[best]).bfloat16()
    C = C.bfloat16()
    b = torch.randn(V, generator=g).bfloat16() if bias else None
    tok = None
    if K is not None:
        tok = torch.randint(0, V, (N, K), generator=g)
        tok[:, 0] = best
        tok[torch.rand(N, K, generator=g) < ignore] = IGNORE
        if N > 4:
            tok[N // 2] = IGNORE
    return tuple(None if t is None else t.to(device) for t in (E, C, b, tok))


def logits64(E, C, bias):
    z = E.double() @ C.double().T
    return z if bias is None else z + bias.double()


def logit_tol(E, C):
    return (E.double().abs() @ C.double().abs().T).amax(1) * 2.0 ** -14


def reference(E, C, bias, tok, T):
    """(logprobs, entropy, p, ln p, wanted) in 64 bits."""
    y = logits64(E, C, bias) / T
    logp = torch.log_softmax(y, 1)
    p = logp.exp()
    wanted = tok != IGNORE
    lp = torch.where(wanted, logp.gather(1, tok.clamp(min=0)), 0.0)
    H = torch.special.entr(p).sum(1) * wanted.any(1)
    return lp, H, p, logp, wanted


def check_logprobs(E, C, bias, tok, T, lp, H):
    rlp, rH, _, _, wanted = reference(E, C, bias, tok, T)
    dz = logit_tol(E, C) / T
    err = (lp.double() - rlp).abs()
    tol = 2 * dz[:, None] + 2.0 ** -18 * (1 + rlp.abs())
    assert (err <= tol).all(), f"logprob off by {(err / tol).max().item():.2f} of the tolerance"
    assert (lp[~wanted] == 0).all()
    errH = (H.double() - rH).abs()
    tolH = 2 * rH * dz + 2.0 ** -18 * (1 + rH)
    assert (errH <= tolH).all(), f"entropy off by {(errH / tolH).max().item():.2f} of the tolerance"
    assert (H[~wanted.any(1)] == 0).all()


SHAPES = [  # N, D, V, K, bias, temperature
    (1, 8, 1, 1, False, 1.0),
    (1, 64, 31, 1, True, 0.7),
    (5, 72, 130, 2, True, 2.0),
    (33, 128, 257, 1, False, 1.0),
    (129, 136, 1000, 3, True, 0.5),
    (256, 128, 4096, 1, False, 1.0),
    (300, 520, 5003, 32, True, 1.3),   # two parts of K, the second of 8 values
    (640, 1032, 20000, 1, False, 1.0),
    (4097, 64, 50257, 1, True, 1.0),   # two groups of row blocks, units of whole tiles
    (1, 4096, 50000, 1, False, 1.0),
]


@pytest.mark.parametrize("N,D,V,K,has_bias,T", SHAPES)
def test_logprobs_and_entropy(device, N, D, V, K, has_bias, T):
    E, C, bias, tok = make(N, D, V, 1000 + N + D + V, device, has_bias, K)
    if K == 1 and N == 1:
        tok[:] = V - 1
    out = L.cce_logprobs(E, C, tok, 0, bias, T, check=True)
    check_logprobs(E, C, bias, tok, T, out[0], out[1])


@pytest.mark.parametrize("N,D,V,has_bias", [(1, 64, 24, False), (3, 128, 1000, True), (130, 72, 4099, True),
                                            (700, 256, 20011, False), (4224, 64, 33000, False)])
@pytest.mark.parametrize("k", [1, 8, 9, 24])
def test_top_alternatives(device, N, D, V, has_bias, k):
    E, C, bias, _ = make(N, D, V, 7 * N + V + k, device, has_bias)
    check_top(E, C, bias, k, 1.0, lce.linear_top_logprobs(E, C, k, bias=bias))


def check_top(E, C, bias, k, T, top, z=None, dz=None):
    z = logits64(E, C, bias) if z is None else z
    dz = logit_tol(E, C) if dz is None else dz
    ids = torch.sort(z, dim=1, descending=True, stable=True)[1][:, :k]
    assert torch.equal(top.ids, ids)
    ref = torch.log_softmax(z / T, 1).gather(1, ids)
    err = (top.logprobs.double() - ref).abs()
    assert (err <= 2 * dz[:, None] / T + 2.0 ** -18 * (1 + ref.abs())).all(), err.max().item()


def test_saved_maxima_of_a_long_batch_with_alternatives(device):
    """Alternatives are found a slab of rows at a time; the maxima saved for the backward are those of all rows."""
    E, C, _, tok = make(4224, 64, 700, 23, device, K=1)
    lp, H, lse, tmax, tl, ti = L.cce_logprobs(E, C, tok, 3, save_max=True, check=True)
    plain = L.cce_logprobs(E, C, tok, save_max=True)
    assert torch.equal(tmax, plain[3])  # (the statistics are added in another order)
    check_logprobs(E, C, None, tok, 1.0, lp, H)
    z = torch.full((4224, 704), -math.inf, dtype=torch.float64, device=device)
    z[:, :700] = logits64(E, C, None)
    most = z.reshape(4224, 11, 64).amax(2).T
    assert ((tmax.reshape(11, 4224).double() - most).abs() <= logit_tol(E, C)).all()


def test_equal_alternatives_go_to_the_lowest_id(device):
    """Rows of C repeated all over the vocabulary, across tiles and segments; a row of E that is zero (every logit
    equal); logits that differ by less than fp32 can tell."""
    N, D, V = 200, 128, 30000
    E, C, _, _ = make(N, D, V, 5, device)
    g = torch.Generator().manual_seed(6)
    spots = torch.randperm(V, generator=g)[:3000].to(device)
    C[spots] = C[spots[:10]].repeat(300, 1)
    E[3] = 0
    E[4] = C[spots[0]] * 8
    for k in (5, 24):
        check_top(E, C, None, k, 1.0, lce.linear_top_logprobs(E, C, k))


def test_close_alternatives_are_ordered_in_64_bits(device):
    """Logits of about 1000 that differ by 2^-16 and less: below the step of fp32 there."""
    D, V = 1024, 2000
    g = torch.Generator().manual_seed(9)
    E = torch.ones(7, D).bfloat16()
    C = torch.randn(V, D, generator=g).bfloat16() * 0.01
    C[100:110] = 1.0
    for i in range(10):  # one entry a little larger, by 2^-7 steps scaled down by the matching entry of E
        C[100 + i, 5] = 1.0 + 2.0 ** -7 * ((3 * i) % 10)
    E[:, 5] = 2.0 ** -12
    E, C = E.to(device), C.to(device)
    check_top(E, C, None, 8, 1.0, lce.linear_top_logprobs(E, C, 8))


def test_masked_columns_and_rows(device):
    """A bias of -inf takes columns out; the type's lowest value leaves them in at probability 0; a row of which
    nothing is left gives -inf, entropy 0 and no gradient."""
    N, D, V = 140, 64, 1500
    E, C, bias, tok = make(N, D, V, 21, device, True, 2)
    bias[::3] = -math.inf
    bias[1::7] = torch.finfo(torch.bfloat16).min
    lp, H, *_ = L.cce_logprobs(E, C, tok, 0, bias, 1.0, check=True)
    z = logits64(E, C, bias)
    ref = torch.log_softmax(z, 1)
    rlp = torch.where(tok != IGNORE, ref.gather(1, tok.clamp(min=0)), 0.0)
    dz = logit_tol(E, C)
    fine = rlp > -1e30
    assert ((lp.double() - rlp).abs()[fine] <= (2 * dz[:, None] + 2.0 ** -18 * (1 + rlp.abs()))[fine]).all()
    assert (lp[~fine] < -1e30).all()
    assert torch.equal(torch.isinf(lp), torch.isinf(rlp.float()))
    rH = torch.special.entr(ref.exp()).sum(1) * (tok != IGNORE).any(1)
    assert ((H.double() - rH).abs() <= 2 * rH * dz + 2.0 ** -18 * (1 + rH)).all()
    # only 5 columns left: the alternatives beyond them are -inf, the lowest ids first
    bias[:] = -math.inf
    bias[700:705] = 0
    top = lce.linear_top_logprobs(E, C, 8, bias=bias)
    z = logits64(E, C, bias)
    assert torch.equal(top.ids, torch.sort(z, dim=1, descending=True, stable=True)[1][:, :8])
    assert torch.isinf(top.logprobs[:, 5:]).all() and torch.isfinite(top.logprobs[:, :5]).all()
    # nothing left
    bias[:] = -math.inf
    e = E.clone().requires_grad_(True)
    c = C.clone().requires_grad_(True)
    out = lce.linear_logprobs(e, c, tok, bias=bias)
    wanted = tok != IGNORE
    assert (out.logprobs[wanted] == -math.inf).all() and (out.logprobs[~wanted] == 0).all() and (out.entropy == 0).all()
    ge, gc = torch.autograd.grad((out.logprobs, out.entropy), (e, c),
                                 (torch.ones_like(out.logprobs), torch.ones_like(out.entropy)))
    assert (ge == 0).all() and (gc == 0).all()
    # every logit at the lowest value: all equal
    bias[:] = torch.finfo(torch.bfloat16).min
    lp, H, *_ = L.cce_logprobs(E, C, tok, 0, bias, 1.0, check=True)
    assert ((lp[wanted] + math.log(V)).abs() <= 2.0 ** -18 * 9).all()
    assert ((H[wanted.any(1)] - math.log(V)).abs() <= 2.0 ** -18 * 9).all()


GRAD_SHAPES = [  # N, D, V, K, bias, T
    (1, 8, 1, 1, False, 1.0),
    (5, 72, 130, 2, True, 2.0),
    (129, 136, 1000, 1, True, 0.5),
    (256, 128, 4096, 1, False, 1.0),
    (300, 520, 5003, 8, True, 1.3),
    (1100, 256, 20000, 32, False, 0.7),
]


def grad_reference(E, C, bias, tok, T, g, h):
    lp, H, p, logp, wanted = reference(E, C, bias, tok, T)
    gw = torch.where(wanted, g.double(), 0.0)
    hw = torch.where(wanted.any(1), h.double(), 0.0)[:, None]
    G = -p * (gw.sum(1, keepdim=True) + hw * (logp + H[:, None])) / T
    mag = p * (gw.sum(1, keepdim=True).abs() + hw.abs() * (logp.abs() + H[:, None])) / T
    at = tok.clamp(min=0)
    dz = (2 * logit_tol(E, C) / T + 2.0 ** -18)[:, None]
    eG = mag * dz + mag * 2.0 ** -20 + p * hw.abs() * dz / T
    G.scatter_add_(1, at, gw / T)
    eG.scatter_add_(1, at, gw.abs() / T * 2.0 ** -22)
    eG += 2.0 ** -8 * G.abs()
    a = G.abs() + eG
    E, C = E.double() * wanted.any(1)[:, None], C.double()
    dE, dC, db = G @ C, G.T @ E, G.sum(0)
    # dC's rows of E carry the rows' scales and are rounded to bf16 with them: 2^-8 more
    tol = (eG @ C.abs() + 2.0 ** -12 * (a @ C.abs()), eG.T @ E.abs() + (2.0 ** -8 + 2.0 ** -12) * (a.T @ E.abs()),
           eG.sum(0) + 2.0 ** -12 * a.sum(0))
    return (dE, dC, db), tol


@pytest.mark.parametrize("N,D,V,K,has_bias,T", GRAD_SHAPES)
@pytest.mark.parametrize("out_fp32", [ops.OUT_FP32, ops.OUT_BF16])
def test_gradients(device, N, D, V, K, has_bias, T, out_fp32):
    E, C, bias, tok = make(N, D, V, 31 + N + V, device, has_bias, K)
    gen = torch.Generator().manual_seed(N + K)
    g = torch.randn(N, K, generator=gen).to(device)
    h = torch.randn(N, generator=gen).to(device)
    lp, H, lse, _, _, _ = L.cce_logprobs(E, C, tok, 0, bias, T, check=True)
    for gg, hh in ((g, h), (g, None), (None, h)):
        out = L.cce_logprobs_backward(E, C, tok, lp, lse, H, None, gg, hh, 0.0, bias, True, T, out_fp32=out_fp32,
                                      check=True)
        ref, tol = grad_reference(E, C, bias, tok, T, torch.zeros_like(g) if gg is None else gg,
                                  torch.zeros_like(h) if hh is None else hh)
        assert out[2].item() == 0
        for name, got, r, t in zip(("dE", "dC", "dbias"), (out[0], out[1], out[3]), ref, tol):
            t = t + 1e-30 + (2.0 ** -8 * (r.abs() + t) if got.dtype == torch.bfloat16 else 0.0)
            worst = ((got.double() - r).abs() / t).max().item()
            assert worst <= 1.0, f"{name}: {worst:.2f} of the tolerance"
        assert (out[0][(tok == IGNORE).all(1)] == 0).all()
