"""Checks of the head operators' arguments that need no GPU: saved statistics, derivatives, odd forms of arguments."""
import ctypes

import pytest
import torch

import linear_cross_entropy_06_b200 as lce
from linear_cross_entropy_06_b200 import logprobs as L
from linear_cross_entropy_06_b200 import ops
from linear_cross_entropy_06_b200.build import build


@pytest.fixture(scope="module")
def lib():
    build()
    return ops.load_library()


def operands(N=4, D=32, V=100):
    return torch.zeros(N, D, dtype=torch.bfloat16), torch.zeros(V, D, dtype=torch.bfloat16)


def test_row_stats_are_checked(lib):
    e, c = operands()
    t = torch.zeros(4, 2, dtype=torch.int64)
    lp, lse, H = torch.zeros(4, 2), torch.zeros(4), torch.zeros(4)
    for bad in (torch.zeros(2, 3), torch.zeros(8), torch.zeros(4, 2).T, torch.zeros(2, 4, dtype=torch.float64)):
        with pytest.raises(lce.CCEError, match="row_stats"):
            L.cce_logprobs(e, c, t, row_stats=bad)
        with pytest.raises(lce.CCEError, match="row_stats"):
            L.cce_logprobs_backward(e, c, t, lp, lse, H, None, lp, H, row_stats=bad)
    with pytest.raises(lce.CCEError, match="given tokens"):
        L.cce_logprobs(e, c, None, 3, row_stats=torch.zeros(2, 4))
    with pytest.raises(lce.CCEError, match="no CPU path"):
        L.cce_logprobs(e, c, t, row_stats=torch.zeros(2, 4))


def test_the_calls_with_statistics_refuse_what_the_plain_ones_do(lib):
    good = ops.LogprobProblem(4, 32, 100, -100, 2, 0, 1.0, 0, 0)
    bad = ops.LogprobProblem(4, 32, 100, -100, 33, 0, 1.0, 0, 0)
    for p, E, size, status in ((bad, 16, 1 << 40, 1), (good, None, 1 << 40, 1), (good, 8, 1 << 40, 1), (good, 16, 0, 3)):
        assert lib.cce_logprobs_stats(ctypes.byref(p), E, 16, None, None, 16, 16, 16, 16, 16, None, None, None, 16,
                                      size, None) == status
        assert lib.cce_logprobs_stats_backward(ctypes.byref(p), E, 16, None, 16, 16, 16, 16, 16, None, 16, 16, 0.0, 16,
                                               16, None, 0, 0, 16, 16, size, None) == status
    assert lib.cce_logprobs_stats_backward(ctypes.byref(good), 16, 16, None, 16, 16, 16, 16, 16, None, 16, 16, 0.0, 16,
                                           16, 16, 0, 2, 16, 16, 1 << 40, None) == 1  # dbias_fp32


def test_forward_mode_derivatives_are_refused(lib):
    """A dual input has no requires_grad: without a refusal the outputs come back without a tangent."""
    from torch.autograd import forward_ad

    e, c = operands()
    bias = torch.zeros(100)
    q = lce.Int8Rows(torch.zeros(100, 32, dtype=torch.int8), torch.ones(100))
    t = torch.zeros(4, dtype=torch.int64)
    with forward_ad.dual_level():
        de, dc, db = (forward_ad.make_dual(x, torch.ones_like(x)) for x in (e, c, bias))
        dq = lce.Int8Rows(q.values, forward_ad.make_dual(q.scale, torch.ones(100)))
        for call in (lambda: lce.linear_logprobs(de, c, t), lambda: lce.linear_logprobs(e, dc, t),
                     lambda: lce.linear_logprobs(e, c, t, bias=db), lambda: lce.linear_logprobs(de, q, t, top_k=2),
                     lambda: lce.linear_logprobs(e, dq, t), lambda: lce.linear_top_logprobs(de, c, 3),
                     lambda: lce.linear_top_logprobs(e, q, 3, bias=db), lambda: lce.quantize_int8(dc),
                     lambda: lce.int8_linear(de, q), lambda: lce.int8_linear(e, dq),
                     lambda: lce.int8_linear(e, q, bias=db)):
            with pytest.raises(NotImplementedError, match="forward-mode"):
                call()
        with pytest.raises(lce.CCEError, match="no CPU path"):  # a level without dual inputs is nothing to refuse
            lce.linear_logprobs(e, c, t, bias=bias)


def test_bad_arguments_are_named_where_they_are_given(lib):
    e, c = operands()
    with pytest.raises(lce.CCEError, match="1 to 32 tokens"):  # none, with more leading dimensions than one
        lce.linear_logprobs(e.reshape(2, 2, 32), c, torch.zeros(2, 2, 0, dtype=torch.int64))
    with pytest.raises(ValueError, match="filter_eps"):  # not first in the backward
        lce.linear_logprobs(e, c, torch.zeros(4, dtype=torch.int64), filter_eps=float("nan"))
