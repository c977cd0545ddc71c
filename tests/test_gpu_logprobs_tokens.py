"""Rows all of whose tokens are out of range: the log-probabilities are NaN, the entropy is not, with its gradient."""
import pytest
import torch

import linear_cross_entropy_06_b200 as lce

from test_gpu_logprobs import IGNORE, grad_reference, make
from test_gpu_logprobs_use import check_grads

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("K", [1, 3])
def test_entropy_of_rows_whose_tokens_are_out_of_range(device, K):
    N, D, V = 140, 64, 700
    E, C, _, tok = make(N, D, V, 40 + K, device, K=K, ignore=0.0)
    tok = tok.clamp(min=0)
    bad = tok.clone()
    bad[::2] = torch.tensor([-1, V, V + 2 ** 40])[:K].to(device)
    bad[7] = IGNORE
    e, c = E.clone().requires_grad_(True), C.clone().requires_grad_(True)
    out = lce.linear_logprobs(e, c, bad)
    assert torch.isnan(out.logprobs[::2]).all() and torch.isfinite(out.entropy).all()
    h = torch.randn(N, generator=torch.Generator().manual_seed(1)).to(device)
    got = torch.autograd.grad(out.entropy, (e, c), h)
    ask = tok.clone()
    ask[7] = IGNORE
    ref, tol = grad_reference(E, C, None, ask, 1.0, torch.zeros(N, K, device=device), h)
    check_grads(got, ref, tol)
    # of the log-probabilities, nothing comes from such tokens
    got = torch.autograd.grad(lce.linear_logprobs(e, c, bad).logprobs, (e, c), torch.ones(N, K, device=device))
    ask[::2] = IGNORE
    ref, tol = grad_reference(E, C, None, ask, 1.0, torch.ones(N, K, device=device), torch.zeros(N, device=device))
    check_grads(got, ref, tol)
