"""Host-side checks of the head operators that need no GPU: sizes, argument validation, refusals."""
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


def problem(N=256, D=128, V=4096, tokens=1, top=0, T=1.0, int8=0, reserved=0):
    return ops.LogprobProblem(N, D, V, -100, tokens, top, T, int8, reserved)


def forward(lib, p, size=1 << 40, **ptr):
    a = dict(E=16, C=16, scale=None, bias=None, tokens=16, lp=16, H=16, lse=16, tmax=None, top=16, ids=16, ws=16)
    a.update(ptr)
    return lib.cce_logprobs(ctypes.byref(p), a["E"], a["C"], a["scale"], a["bias"], a["tokens"], a["lp"], a["H"],
                            a["lse"], a["tmax"], a["top"], a["ids"], a["ws"], size, None)


def backward(lib, p, size=1 << 40, eps=0.0, out=0, **ptr):
    a = dict(E=16, C=16, bias=None, tokens=16, lp=16, lse=16, H=16, tmax=None, g=16, h=16, dE=16, dC=16, db=None,
             filt=16, ws=16)
    a.update(ptr)
    return lib.cce_logprobs_backward(ctypes.byref(p), a["E"], a["C"], a["bias"], a["tokens"], a["lp"], a["lse"],
                                     a["H"], a["tmax"], a["g"], a["h"], eps, a["dE"], a["dC"], a["db"], out,
                                     a["filt"], a["ws"], size, None)


@pytest.mark.parametrize("bad", [dict(N=-1), dict(D=0), dict(D=12), dict(V=0), dict(tokens=33), dict(tokens=-1),
                                 dict(top=25), dict(top=-1), dict(tokens=0), dict(V=3, top=4), dict(T=0.0),
                                 dict(T=-1.0), dict(T=float("nan")), dict(T=float("inf")), dict(T=1e-7), dict(T=1e7),
                                 dict(reserved=1), dict(int8=2), dict(int8=1, D=24), dict(int8=1, D=131088),
                                 dict(V=1 << 31)])
def test_bad_problems_are_refused(lib, bad):
    p = problem(**bad)
    assert lib.cce_logprobs_workspace_size(ctypes.byref(p)) == 0
    assert forward(lib, p, scale=16) == 1
    assert lib.cce_last_error_message()
    assert lib.cce_logprobs_backward_workspace_size(ctypes.byref(p), 0) == 0
    assert backward(lib, p) == 1


@pytest.mark.parametrize("ptr", [dict(E=None), dict(C=None), dict(tokens=None), dict(lp=None), dict(H=None),
                                 dict(lse=None), dict(ws=None), dict(E=8), dict(C=24), dict(bias=8), dict(ws=8)])
def test_missing_and_misaligned_pointers_are_refused(lib, ptr):
    assert forward(lib, problem(), **ptr) == 1


def test_alternatives_need_their_outputs_and_8_bit_rows_their_scales(lib):
    assert forward(lib, problem(top=4), top=None) == 1
    assert forward(lib, problem(top=4), ids=None) == 1
    assert forward(lib, problem(int8=1)) == 1
    assert b"NULL" in lib.cce_last_error_message()


def test_small_workspaces_are_refused(lib):
    p = problem(top=4)
    need = lib.cce_logprobs_workspace_size(ctypes.byref(p))
    assert need > 0 and forward(lib, p, size=need - 1) == 3
    need = lib.cce_logprobs_backward_workspace_size(ctypes.byref(p), 0)
    assert need > 0 and backward(lib, p, size=need - 1) == 3
    need = lib.cce_int8_linear_workspace_size(100, 64, 1000)
    assert need >= 100 * 64
    assert lib.cce_int8_linear(100, 64, 1000, 16, 16, 16, None, 32, 0, 16, need - 1, None) == 3


@pytest.mark.parametrize("ptr", [dict(E=None), dict(dE=None), dict(dC=None), dict(lp=None), dict(lse=None),
                                 dict(filt=None), dict(H=None), dict(db=8), dict(dE=8)])
def test_backward_pointers(lib, ptr):
    assert backward(lib, problem(), **ptr) == 1


def test_backward_refusals(lib):
    assert backward(lib, problem(), eps=float("nan")) == 1
    assert backward(lib, problem(), eps=0.5) == 1  # skipping needs the saved maxima
    assert backward(lib, problem(), out=3) == 1
    assert backward(lib, problem(int8=1)) == 1
    assert b"no gradient" in lib.cce_last_error_message()
    assert backward(lib, problem(tokens=0, top=4)) == 1


def test_int8_refusals(lib):
    assert lib.cce_int8_linear_workspace_size(4, 24, 100) == 0
    assert lib.cce_int8_linear(4, 24, 100, 16, 16, 16, None, 16, 0, 16, 1 << 30, None) == 1
    assert lib.cce_int8_linear(4, 32, 100, 16, 16, None, None, 16, 0, 16, 1 << 30, None) == 1
    assert lib.cce_int8_linear(4, 32, 100, 16, 16, 16, None, 16, 2, 16, 1 << 30, None) == 1
    assert lib.cce_int8_linear(4, 32, 100, 16, 16, 16, None, 24, 0, 16, 1 << 30, None) == 1
    assert lib.cce_quantize_int8(16, 4, 24, 16, 16, None) == 1
    assert lib.cce_quantize_int8(None, 4, 32, 16, 16, None) == 1
    assert lib.cce_quantize_int8(24, 4, 32, 16, 16, None) == 1


def test_workspaces_stay_far_below_the_logits(lib):
    """Long batches: the alternatives are found a slab of rows at a time, the statistics are a few floats a segment."""
    logits = 32768 * 128256 * 2
    for top in (0, 24):
        p = problem(N=32768, D=4096, V=128256, tokens=1, top=top)
        assert lib.cce_logprobs_workspace_size(ctypes.byref(p)) < logits // 30
    assert lib.cce_logprobs_backward_workspace_size(ctypes.byref(p), 0) < logits // 4 + 32768 * 4096 * 2


def operands(N=4, D=32, V=100, dtype=torch.bfloat16):
    return torch.zeros(N, D, dtype=dtype), torch.zeros(V, D, dtype=torch.bfloat16)


def test_python_refuses_wrong_types_and_shapes(lib):
    e, c = operands()
    t = torch.zeros(4, dtype=torch.int64)
    with pytest.raises(lce.CCEError, match="bfloat16"):
        lce.linear_logprobs(e.float(), c, t)
    with pytest.raises(lce.CCEError, match="bfloat16"):
        lce.linear_logprobs(e, c.half(), t)
    with pytest.raises(lce.CCEError, match=r"must be \[V, 32\]"):
        lce.linear_logprobs(e, c[:, :16], t)
    with pytest.raises(ValueError, match="tokens shape"):
        lce.linear_logprobs(e, c, t[:3])
    with pytest.raises(lce.CCEError, match="1 to 32 tokens"):
        lce.linear_logprobs(e, c, torch.zeros(4, 33, dtype=torch.int64))
    with pytest.raises(lce.CCEError, match="1 to 32 tokens"):
        lce.linear_logprobs(e, c, torch.zeros(4, 0, dtype=torch.int64))
    for T in (0.0, -1.0, 1e-7, 1e7, float("nan")):
        with pytest.raises(ValueError, match="temperature"):
            lce.linear_logprobs(e, c, t, temperature=T)
    with pytest.raises(ValueError, match="alternatives"):
        lce.linear_logprobs(e, c, t, top_k=25)
    with pytest.raises(ValueError, match="alternatives"):
        lce.linear_top_logprobs(e, c[:3], 4)
    with pytest.raises(ValueError, match="at least 1"):
        lce.linear_top_logprobs(e, c, 0)
    with pytest.raises(ValueError, match="shift"):
        lce.linear_logprobs(e, c, torch.zeros(4, 2, dtype=torch.int64), shift=True)
    with pytest.raises(lce.CCEError, match="int64"):
        L.cce_logprobs(e, c, t[:, None].int())
    with pytest.raises(lce.CCEError, match="no CPU path"):
        lce.linear_logprobs(e, c, t)
    with pytest.raises(lce.CCEError, match="no CPU path"):
        lce.linear_top_logprobs(e, c, 4)


def test_python_refuses_bad_8_bit_rows(lib):
    e, c = operands()
    q = lce.Int8Rows(torch.zeros(100, 32, dtype=torch.int8), torch.ones(100))
    t = torch.zeros(4, dtype=torch.int64)
    with pytest.raises(lce.CCEError, match="Int8Rows"):
        lce.int8_linear(e, c)
    with pytest.raises(lce.CCEError, match="int8"):
        lce.int8_linear(e, lce.Int8Rows(c, q.scale))
    with pytest.raises(lce.CCEError, match="100 entries"):
        lce.int8_linear(e, lce.Int8Rows(q.values, q.scale[:99]))
    with pytest.raises(lce.CCEError, match="float32"):
        lce.int8_linear(e, lce.Int8Rows(q.values, q.scale.double()))
    with pytest.raises(lce.CCEError, match="multiple of 16"):
        lce.int8_linear(e[:, :24].contiguous(), lce.Int8Rows(q.values[:, :24], q.scale))
    with pytest.raises(lce.CCEError, match="out_dtype"):
        lce.int8_linear(e, q, out_dtype=torch.float16)
    with pytest.raises(ValueError, match="no gradient"):
        lce.linear_logprobs(e.requires_grad_(True), q, t)
    with pytest.raises(lce.CCEError, match="multiple of 16"):
        lce.quantize_int8(torch.zeros(4, 24, dtype=torch.bfloat16))
    with pytest.raises(lce.CCEError, match="bfloat16"):
        lce.quantize_int8(torch.zeros(4, 32))
    with pytest.raises(lce.CCEError, match="no CPU path"):
        lce.quantize_int8(torch.zeros(4, 32, dtype=torch.bfloat16))


def test_backward_checks_the_saved_state(lib):
    e, c = operands()
    t = torch.zeros(4, 2, dtype=torch.int64)
    lp, lse, H = torch.zeros(4, 2), torch.zeros(4), torch.zeros(4)
    with pytest.raises(lce.CCEError, match="lse"):
        L.cce_logprobs_backward(e, c, t, lp, lse[:3], H, None, None, None)
    with pytest.raises(lce.CCEError, match="logprobs"):
        L.cce_logprobs_backward(e, c, t, lp[:, :1], lse, H, None, None, None)
    with pytest.raises(lce.CCEError, match="grad_entropy"):
        L.cce_logprobs_backward(e, c, t, lp, lse, H, None, None, H.double())
    with pytest.raises(lce.CCEError, match="tile_max"):
        L.cce_logprobs_backward(e, c, t, lp, lse, H, None, lp, None, filter_eps=0.1)
    with pytest.raises(lce.CCEError, match="no CPU path"):
        L.cce_logprobs_backward(e, c, t, lp, lse, H, None, lp, H)
