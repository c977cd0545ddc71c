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
    with pytest.raises(lce.CCEError, match="no CPU path"):
        L.cce_logprobs(e, c, t, row_stats=torch.zeros(2, 4))


def test_the_calls_with_statistics_refuse_what_the_plain_ones_do(lib):
    good = ops.LogprobProblem(4, 32, 100, -100, 2, 0, 1.0, 0, 0)
    bad = ops.LogprobProblem(4, 32, 100, -100, 33, 0, 1.0, 0, 0)
    for p, E, size, status in ((bad, 16, 1 << 40, 1), (good, None, 1 << 40, 1), (good, 8, 1 << 40, 1), (good, 16, 0, 3)):
        assert lib.cce_logprobs_stats(ctypes.byref(p), E, 16, None, None, 16, 16, 16, 16, 16, None, None, None, 16,
                                      size, None) == status
        assert lib.cce_logprobs_stats_backward(ctypes.byref(p), E, 16, None, 16, 16, 16, 16, 16, None, 16, 16, 0.0, 16,
                                               16, None, 0, 16, 16, size, None) == status
