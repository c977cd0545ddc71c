"""The head operators as a program uses them: through autograd, with leading dimensions, shifted, strided and shared
inputs, on other streams, captured into graphs, with padding that holds NaN, skipping, errors, and one after another."""
import math
import os
import subprocess
import sys

import pytest
import torch

import linear_cross_entropy_06_b200 as lce
from linear_cross_entropy_06_b200 import logprobs as L
from linear_cross_entropy_06_b200 import ops

from test_gpu_logprobs import (IGNORE, check_logprobs, check_top, grad_reference, logit_tol, logits64, make, reference)

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def check_grads(got, ref, tol):
    for name, x, r, t in zip(("dE", "dC", "dbias"), got, ref, tol):
        t = t + 1e-30 + (2.0 ** -8 * (r.abs() + t) if x.dtype == torch.bfloat16 else 0.0)
        worst = ((x.double().reshape(r.shape) - r).abs() / t).max().item()
        assert worst <= 1.0, f"{name}: {worst:.2f} of the tolerance"


@pytest.mark.parametrize("K", [None, 3])
def test_autograd_with_leading_dimensions(device, K):
    E, C, bias, tok = make(60, 128, 3000, 1, device, True, K or 1)
    T = 0.8
    e = E.reshape(3, 20, 128).requires_grad_(True)
    c = C.clone().requires_grad_(True)
    b = bias.float().requires_grad_(True)  # a bias of another type gets its gradient in that type
    t = tok.reshape(3, 20, K) if K else tok.reshape(3, 20)
    out = lce.linear_logprobs(e, c, t, bias=b, temperature=T, top_k=4)
    assert out.logprobs.shape == t.shape and out.entropy.shape == (3, 20)
    assert out.top_ids.shape == out.top_logprobs.shape == (3, 20, 4)
    assert not out.top_logprobs.requires_grad and not out.top_ids.requires_grad
    check_logprobs(E, C, bias, tok, T, out.logprobs.reshape(60, -1), out.entropy.reshape(60))
    check_top(E, C, bias, 4, T, lce.TopLogprobs(out.top_logprobs.reshape(60, 4), out.top_ids.reshape(60, 4)))
    gen = torch.Generator().manual_seed(2)
    g = torch.randn(60, K or 1, generator=gen).to(device)
    # both outputs, the entropy by one shared gradient (expanded: strides 0)
    h = torch.full((), 0.3, device=device).expand(3, 20)
    grads = torch.autograd.grad((out.logprobs, out.entropy), (e, c, b), (g.reshape(t.shape), h), retain_graph=True)
    assert grads[0].shape == e.shape and grads[2].dtype == torch.float32
    ref, tol = grad_reference(E, C, bias, tok, T, g, h.reshape(60))
    # the bias's gradient is formed in bf16 first
    tol = (tol[0], tol[1], tol[2] + 2.0 ** -8 * (ref[2].abs() + tol[2]))
    check_grads(grads, ref, tol)
    # one output only
    grads = torch.autograd.grad(out.entropy.sum(), (e, c))
    ref, tol = grad_reference(E, C, bias, tok, T, torch.zeros_like(g), torch.ones(60, device=device))
    check_grads(grads, ref, tol)


def test_gradients_against_differences(device):
    """Along random directions, (f(E + u) - f(E - u)) / 2 of the kernel's own outputs against its gradient. E is a
    multiple of 1/8 within 4 and u of 1/16 within 1/16, so that E + u and E - u are bf16 numbers; what the central
    difference itself is off (its cubic term) is taken from the same quotient in 64 bits."""
    N, D, V, K = 40, 128, 700, 2
    g = torch.Generator().manual_seed(3)
    E = (torch.randint(-32, 33, (N, D), generator=g) / 8.0)
    C = (torch.randn(V, D, generator=g) / math.sqrt(D)).bfloat16().to(device)
    tok = torch.randint(0, V, (N, K), generator=g).to(device)
    w = torch.randn(N, K, generator=g).to(device)
    h = torch.randn(N, generator=g).to(device)
    E = E.bfloat16().to(device)

    def f(x):
        lp, H, *_ = L.cce_logprobs(x, C, tok)
        return (lp.double() * w.double()).sum(1) + H.double() * h.double()

    def f64(x):
        lp, H, *_ = reference(x, C, None, tok, 1.0)
        return (lp * w.double()).sum(1) + H * h.double()

    lp, H, lse, *_ = L.cce_logprobs(E, C, tok)
    dE = L.cce_logprobs_backward(E, C, tok, lp, lse, H, None, w, h, out_fp32=ops.OUT_FP32)[0].double()
    (ref, *_), (tol, *_) = grad_reference(E, C, None, tok, 1.0, w, h)
    dz = logit_tol(E, C)
    f_tol = (w.double().abs() * (2 * dz[:, None] + 2.0 ** -18 * (1 + lp.double().abs()))).sum(1) + \
        h.double().abs() * (2 * H.double() * dz + 2.0 ** -18 * (1 + H.double()))
    for seed in range(4):
        u = (torch.randint(-1, 2, (N, D), generator=torch.Generator().manual_seed(seed)) / 16.0).to(device)
        plus, minus = (E.float() + u).bfloat16(), (E.float() - u).bfloat16()
        assert torch.equal(plus.float() - u, E.float()) and torch.equal(minus.float() + u, E.float())
        quotient = (f(plus) - f(minus)) / 2
        cubic = ((f64(plus) - f64(minus)) / 2 - (ref * u.double()).sum(1)).abs()
        allowed = cubic + f_tol + (tol * u.double().abs()).sum(1)
        assert ((quotient - (dE * u.double()).sum(1)).abs() <= allowed).all()


def test_shift(device):
    E, C, _, tok = make(64, 64, 500, 4, device, K=1, ignore=0.0)
    e, t = E.reshape(4, 16, 64), tok.reshape(4, 16).clamp(min=0)
    out = lce.linear_logprobs(e, C, t, shift=True, top_k=1)
    assert out.logprobs.shape == (4, 15) and out.entropy.shape == (4, 15) and out.top_ids.shape == (4, 15, 1)
    ref = torch.log_softmax(logits64(E, C, None), 1).reshape(4, 16, -1)[:, :-1].gather(2, t[:, 1:, None])[..., 0]
    dz = logit_tol(E, C).reshape(4, 16)[:, :-1]
    assert ((out.logprobs.double() - ref).abs() <= 2 * dz + 2.0 ** -18 * (1 + ref.abs())).all()


def test_padding_that_holds_nan_reaches_nothing(device):
    """Rows that ask for nothing may hold anything; the gradients of the others are what they would be without."""
    N, D, V = 300, 136, 2000
    E, C, bias, tok = make(N, D, V, 5, device, True, 2)
    pad = torch.zeros(N, dtype=torch.bool, device=device)
    pad[-45:] = True
    pad[130:140] = True
    tok[pad] = IGNORE
    g, h = torch.randn(N, 2, device=device), torch.randn(N, device=device)
    results = []
    for fill in (0.0, math.nan, math.inf):
        x = E.clone()
        x[pad] = fill
        lp, H, lse, *_ = L.cce_logprobs(x, C, tok, 0, bias, check=True)
        gg, hh = g.clone(), h.clone()
        gg[pad], hh[pad] = math.nan, math.nan  # nor are their gradients read into anything
        out = L.cce_logprobs_backward(x, C, tok, lp, lse, H, None, gg, hh, 0.0, bias, True, check=True)
        assert (lp[pad] == 0).all() and (H[pad] == 0).all()
        assert (out[0][pad].view(torch.int16) == 0).all()
        results.append((lp, H, out[0], out[1], out[3]))
    for other in results[1:]:
        assert torch.equal(other[0], results[0][0]) and torch.equal(other[1], results[0][1])
        for a, b in zip(other[2:], results[0][2:]):
            assert torch.isfinite(a.float()).all()
            assert ((a.float() - b.float()).norm() <= 1e-3 * b.float().norm())  # dE and dbias: order of fp32 adds


def test_a_row_with_nan_stays_alone(device):
    E, C, _, tok = make(200, 64, 1500, 6, device, K=1, ignore=0.0)
    tok = tok.clamp(min=0)
    clean = L.cce_logprobs(E, C, tok, 5)
    x = E.clone()
    x[77, 3] = math.nan
    out = L.cce_logprobs(x, C, tok, 5)
    assert torch.isnan(out[0][77]).all() and torch.isnan(out[1][77]) and torch.isnan(out[4][77]).all()
    assert ((out[5][77] >= -1) & (out[5][77] < 1500)).all()
    keep = torch.arange(200, device=device) != 77
    for a, b in zip((out[0], out[1], out[4], out[5]), (clean[0], clean[1], clean[4], clean[5])):
        assert torch.equal(a[keep], b[keep])


def test_same_token_twice_and_order_of_tokens(device):
    E, C, _, tok = make(50, 64, 900, 7, device, K=4, ignore=0.0)
    tok = tok.clamp(min=0)
    tok[:, 1] = tok[:, 0]
    lp, H, lse, *_ = L.cce_logprobs(E, C, tok)
    assert torch.equal(lp[:, 0], lp[:, 1])
    g = torch.randn(50, 4, device=device)
    out = L.cce_logprobs_backward(E, C, tok, lp, lse, H, None, g, None, out_fp32=ops.OUT_FP32)
    ref, tol = grad_reference(E, C, None, tok, 1.0, g, torch.zeros(50, device=device))
    check_grads(out[:2], ref, tol)


@pytest.mark.parametrize("K", [1, 6])
def test_skipping_keeps_tokens_and_drops_the_rest(device, K):
    """filter_eps: units of 128 rows x 64 columns whose probabilities are all below it add nothing, except units that
    hold a given token."""
    N, D, V, eps = 400, 256, 9000, 2.0 ** -12
    E, C, bias, tok = make(N, D, V, 8, device, True, K, alpha=20.0)
    bias = bias * 0.25
    T = 1.0
    g, h = torch.randn(N, K, device=device), torch.randn(N, device=device)
    lp, H, lse, tmax, _, _ = L.cce_logprobs(E, C, tok, 0, bias, T, save_max=True, check=True)
    out = L.cce_logprobs_backward(E, C, tok, lp, lse, H, tmax, g, h, eps, bias, True, T, out_fp32=ops.OUT_FP32,
                                  check=True)
    y = logits64(E, C, bias)
    wanted = tok != IGNORE
    p = torch.softmax(y, 1) * wanted.any(1)[:, None]
    nb, nt = -(-N // 128), -(-V // 64)
    grid = torch.zeros(nb * 128, nt * 64, dtype=torch.float64, device=device)
    grid[:N, :V] = p
    most = grid.reshape(nb, 128, nt, 64).amax((1, 3))
    assert not ((most / eps - 1).abs() < 1e-3).any(), "an unlucky seed: a unit lies on the border"
    held = torch.zeros(nb, nt, dtype=torch.bool, device=device)
    rows = torch.arange(N, device=device)[:, None].expand(N, K)[wanted]
    held[rows // 128, tok[wanted] // 64] = True
    keep = (most >= eps) | held
    assert out[2].item() == int((~keep).sum()) > 0
    keep = keep.repeat_interleave(128, 0)[:N].repeat_interleave(64, 1)[:, :V]
    gw = torch.where(wanted, g.double(), 0.0)
    hw = torch.where(wanted.any(1), h.double(), 0.0)[:, None]
    logp = torch.log_softmax(y, 1)
    G = -p * (gw.sum(1, keepdim=True) + hw * (logp + torch.special.entr(p).sum(1)[:, None]))
    G = (G * keep).scatter_add_(1, tok.clamp(min=0), gw)
    (dE, dC, db), tol = grad_reference(E, C, bias, tok, T, g, h)
    E64 = E.double() * wanted.any(1)[:, None]
    check_grads((out[0], out[1], out[3]), (G @ C.double(), G.T @ E64, G.sum(0)), tol)


def test_strided_and_misaligned_inputs(device):
    E, C, bias, tok = make(70, 64, 1000, 9, device, True, 2)
    ref = L.cce_logprobs(E, C, tok, 3, bias)
    wide = torch.zeros(70, 200, dtype=torch.bfloat16, device=device)
    wide[:, 3:67] = E
    ct = C.T.contiguous().T  # columns contiguous
    flat = torch.zeros(1000 * 64 + 1, dtype=torch.bfloat16, device=device)
    flat[1:] = C.reshape(-1)
    b = torch.zeros(1001, dtype=torch.bfloat16, device=device)
    b[1:] = bias
    tt = tok.T.contiguous().T
    for x, y, z, t in ((wide[:, 3:67], ct, b[1:], tt), (E, flat[1:].view(1000, 64), bias.expand(1000), tok)):
        out = L.cce_logprobs(x, y, t, 3, z)
        for a, r in zip(out, ref):
            assert a is None or torch.equal(a, r)
    g = torch.randn(2, 70, device=device).T
    lp, H, lse = ref[:3]
    a = L.cce_logprobs_backward(wide[:, 3:67], ct, tt, lp, lse, H, None, g, None, 0.0, b[1:], True)
    r = L.cce_logprobs_backward(E, C, tok, lp, lse, H, None, g.contiguous(), None, 0.0, bias, True)
    assert torch.equal(a[1], r[1])


@pytest.mark.parametrize("N", [0, 1])
def test_no_rows_and_one(device, N):
    C = torch.randn(50, 64, device=device).bfloat16()
    e = torch.randn(2, N, 64, device=device).bfloat16().requires_grad_(True)
    c = C.clone().requires_grad_(True)
    out = lce.linear_logprobs(e, c, torch.zeros(2, N, dtype=torch.int64, device=device), top_k=3)
    assert out.logprobs.shape == (2, N) and out.top_ids.shape == (2, N, 3)
    (out.logprobs.sum() + out.entropy.sum()).backward()
    assert e.grad.shape == e.shape and c.grad.shape == c.shape
    if N == 0:
        assert (c.grad == 0).all()
    q = lce.quantize_int8(C)
    assert lce.int8_linear(e, q).shape == (2, N, 50)
    assert lce.linear_top_logprobs(e, q, 2).ids.shape == (2, N, 2)


def test_rows_behind_the_last_are_left_as_they_were(device):
    """The outputs of a call end where its rows end."""
    lib = ops.load_library()
    import ctypes
    N, D, V, K, k = 37, 64, 500, 2, 5
    E, C, _, tok = make(N, D, V, 10, device, K=K)
    p = ops.LogprobProblem(N, D, V, IGNORE, K, k, 1.0, 0, 0)
    size = lib.cce_logprobs_workspace_size(ctypes.byref(p))
    ws = torch.empty(size + 64, dtype=torch.uint8, device=device).fill_(0xAB)
    f = lambda n: torch.full((n + 8,), 7.0, device=device)
    lp, H, lse, tl = f(N * K), f(N), f(N), f(N * k)
    ids = torch.full((N * k + 8,), 7, dtype=torch.int64, device=device)
    st = lib.cce_logprobs(ctypes.byref(p), E.data_ptr(), C.data_ptr(), None, None, tok.data_ptr(), lp.data_ptr(),
                          H.data_ptr(), lse.data_ptr(), None, tl.data_ptr(), ids.data_ptr(), ws.data_ptr(), size,
                          torch.cuda.current_stream(device).cuda_stream)
    assert st == 0
    torch.cuda.synchronize()
    for t, n in ((lp, N * K), (H, N), (lse, N), (tl, N * k), (ids, N * k)):
        assert (t[n:] == 7).all() and not (t[:n] == 7).all()
    assert (ws[size:] == 0xAB).all()


def test_side_stream_and_two_calls_at_once(device):
    """Calls on two streams at a time: each has its own workspace."""
    cases = [make(200 + 50 * i, 128, 5000, 11 + i, device, K=1) for i in range(4)]
    want = [L.cce_logprobs(E, C, tok, 4) for E, C, _, tok in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    got = []
    for _ in range(3):
        got = []
        for s, (E, C, _, tok) in zip(streams, cases):
            with torch.cuda.stream(s):
                got.append(L.cce_logprobs(E, C, tok, 4))
        torch.cuda.synchronize()
    for a, b in zip(got, want):
        for x, y in zip(a, b):
            assert y is None or torch.equal(x, y)


def test_graph_replay(device):
    """Forward with alternatives, backward and the 8-bit product captured into two graphs and replayed in turn with
    new inputs in place."""
    N, D, V, K = 300, 256, 8000, 2
    E, C, bias, tok = make(N, D, V, 12, device, True, K)
    g, h = torch.randn(N, K, device=device), torch.randn(N, device=device)
    q = lce.quantize_int8(C)

    def step():
        lp, H, lse, _, tl, ti = L.cce_logprobs(E, C, tok, 6, bias)
        dE, dC, _, db = L.cce_logprobs_backward(E, C, tok, lp, lse, H, None, g, h, 0.0, bias, True)
        return lp, H, tl, ti, dC, dE, db

    def serve():
        return (lce.int8_linear(E, q, bias=bias), *lce.linear_top_logprobs(E, q, 3, bias=bias))

    graphs, outs = [], []
    for fn in (step, serve):
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            fn()
        torch.cuda.current_stream().wait_stream(side)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(fn())
        graphs.append(graph)
    for seed in (13, 14):
        E2, _, _, tok2 = make(N, D, V, seed, device, True, K)
        E.copy_(E2)
        tok.copy_(tok2)
        for graph in graphs:
            graph.replay()
        torch.cuda.synchronize()
        a, b = step(), serve()
        for x, y in zip(outs[0][:5], a[:5]):
            assert torch.equal(x, y)
        for x, y in zip(outs[0][5:], a[5:]):  # dE and dbias: the order of fp32 adds is not fixed
            assert (x.float() - y.float()).norm() <= 1e-3 * y.float().norm()
        for x, y in zip(outs[1], b):
            assert torch.equal(x, y)


def test_autograd_captured(device):
    """Forward and backward through autograd inside a capture. (No eager graph of the same leaves may be alive then:
    torch ties a leaf's gradient to the stream of the graph that used it first, and refuses the capture.)"""
    E, C, _, tok = make(64, 64, 700, 15, device, K=1, ignore=0.0)
    e, c = E.clone().requires_grad_(True), C.clone().requires_grad_(True)
    t = tok.clamp(min=0)[:, 0]

    def loss():
        out = lce.linear_logprobs(e, c, t)
        return out.logprobs.sum() + 0.1 * out.entropy.sum()

    want = torch.autograd.grad(loss(), (e, c))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        torch.autograd.grad(loss(), (e, c))
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = torch.autograd.grad(loss(), (e, c))
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(got[1], want[1])
    assert (got[0].float() - want[0].float()).norm() <= 1e-3 * want[0].float().norm()


def test_token_out_of_range_is_nan_and_reported(device):
    E, C, _, tok = make(20, 64, 300, 16, device, K=2, ignore=0.0)
    tok = tok.clamp(min=0)
    ref = L.cce_logprobs(E, C, tok)
    bad = tok.clone()
    bad[3, 1], bad[5, 0] = 300, -7
    with pytest.raises(lce.CCEError) as err:
        L.cce_logprobs(E, C, bad, check=True)
    assert err.value.status == 4  # CCE_ERR_TARGET_RANGE
    lp, H, lse, *_ = L.cce_logprobs(E, C, bad)
    hit = bad != tok
    assert torch.isnan(lp[hit]).all() and torch.equal(lp[~hit], ref[0][~hit]) and torch.equal(H, ref[1])
    # the backward reads nothing at such a token
    g = torch.randn(20, 2, device=device)
    out = L.cce_logprobs_backward(E, C, bad, lp, lse, H, None, g, None, check=True)
    skip = tok.clone()
    skip[hit] = IGNORE
    same = L.cce_logprobs_backward(E, C, skip, lp, lse, H, None, g, None)
    assert torch.equal(out[1], same[1])


CHILD = r"""
import os, sys
sys.path.insert(0, os.environ["CCE_ROOT"])
import torch
import linear_cross_entropy_06_b200 as lce
from linear_cross_entropy_06_b200 import logprobs as L
g = torch.Generator().manual_seed(1)
E = torch.randn(200, 128, generator=g).bfloat16().cuda()
C = torch.randn(3000, 128, generator=g).bfloat16().cuda()
t = torch.zeros(200, 1, dtype=torch.int64).cuda()
ref = L.cce_logprobs(E, C, t, 3, check=True)
os.environ["CCE_TEST_INJECT_STALL"] = "4"
try:
    L.cce_logprobs(E, C, t, 3, check=True)
    print("NO-ERROR")
except lce.CCEError as e:
    print("STATUS", e.status)
lp, H, lse, _, tl, ti = L.cce_logprobs(E, C, t, 3)
torch.cuda.synchronize()
print("NAN", all(bool(torch.isnan(x).all()) for x in (lp, H, lse, tl)) and bool((ti == -1).all()))
try:
    lce.int8_linear(E, lce.quantize_int8(C), check=True)
    print("NO-ERROR")
except lce.CCEError as e:
    print("STATUS8", e.status)
os.environ["CCE_TEST_INJECT_STALL"] = "0"
got = L.cce_logprobs(E, C, t, 3, check=True)
print("RECOVERED", all(x is None or torch.equal(x, y) for x, y in zip(got, ref)))
"""


def test_a_wait_that_runs_out_is_reported_and_the_context_survives():
    env = dict(os.environ, CCE_ROOT=ROOT, CCE_WAIT_TIMEOUT_MS="200")
    out = subprocess.run([sys.executable, "-c", CHILD], env=env, capture_output=True, text=True, timeout=300)
    assert out.returncode == 0, out.stderr[-2000:]
    assert "STATUS 5" in out.stdout and "STATUS8 5" in out.stdout, out.stdout  # CCE_ERR_DEVICE_TIMEOUT
    assert "NAN True" in out.stdout and "RECOVERED True" in out.stdout, out.stdout


@pytest.mark.parametrize("T", [2e-6, 1e-3, 1e6])
def test_extreme_temperatures(device, T):
    """Nearly one-hot and nearly flat distributions: finite outputs and gradients."""
    E, C, bias, tok = make(50, 64, 900, 24, device, True, 2)
    bias[7] = -math.inf
    lp, H, lse, _, tl, ti = L.cce_logprobs(E, C, tok, 3, bias, T, check=True)
    ref = torch.log_softmax(logits64(E, C, bias) / T, 1)
    wanted = (tok != IGNORE) & (tok != 7)
    want = ref.gather(1, tok.clamp(min=0))
    dz = (logit_tol(E, C) / T)[:, None]
    assert ((lp.double() - want).abs() <= 2 * dz + 2.0 ** -18 * (1 + want.abs()))[wanted].all()
    rH = torch.special.entr(ref.exp()).sum(1)[wanted.any(1)]
    if T >= 1:
        assert ((H.double()[wanted.any(1)] - rH).abs() <= 2.0 ** -18 * (1 + rH)).all()
    assert torch.isfinite(H).all() and (H >= 0).all() and (H <= math.log(900) + 1e-4).all()
    assert torch.equal(ti, torch.sort(logits64(E, C, bias), dim=1, descending=True, stable=True)[1][:, :3])
    g, h = torch.randn(50, 2, device=device), torch.randn(50, device=device)
    out = L.cce_logprobs_backward(E, C, tok, lp, lse, H, None, g, h, 0.0, bias, True, T, check=True)
    assert all(torch.isfinite(x.float()).all() for x in (out[0], out[1], out[3]))


def test_one_vector(device):
    """e without leading dimensions."""
    E, C, _, tok = make(1, 64, 300, 25, device, K=1, ignore=0.0)
    out = lce.linear_logprobs(E[0], C, tok[0, 0], top_k=2)
    assert out.logprobs.shape == () and out.entropy.shape == () and out.top_ids.shape == (2,)
    many = lce.linear_logprobs(E[0], C, tok[0])
    assert many.logprobs.shape == (1,) and many.logprobs[0] == out.logprobs
    assert lce.linear_top_logprobs(E[0], C, 2).ids.tolist() == out.top_ids.tolist()
    assert lce.int8_linear(E[0], lce.quantize_int8(C)).shape == (300,)


def test_second_derivatives_are_refused(device):
    E, C, _, tok = make(20, 64, 300, 26, device, K=1, ignore=0.0)
    e = E.clone().requires_grad_(True)
    out = lce.linear_logprobs(e, C, tok[:, 0])
    (ge,) = torch.autograd.grad(out.logprobs.sum(), e, create_graph=True)
    with pytest.raises(RuntimeError):
        ge.float().sum().backward()


def test_results_do_not_depend_on_the_batch(device):
    """A row's alternatives are the same alone, in a small batch and in a large one (other splits of the work, grouped
    and ungrouped picks)."""
    E, C, bias, _ = make(1500, 256, 20000, 17, device, True)
    big = lce.linear_top_logprobs(E, C, 12, bias=bias)
    for n in (1, 30, 65, 300):
        part = lce.linear_top_logprobs(E[700:700 + n], C, 12, bias=bias)
        assert torch.equal(part.ids, big.ids[700:700 + n])
        assert (part.logprobs - big.logprobs[700:700 + n]).abs().max() <= 2.0 ** -18 * 24


def test_popular_alternatives(device):
    """Every row wants the same picks: more rows than a work item holds."""
    N, D, V = 900, 64, 6000
    E, C, bias, _ = make(N, D, V, 18, device, True)
    bias[:] = 0
    bias[3000:3040] = 30
    check_top(E, C, bias, 20, 1.0, lce.linear_top_logprobs(E, C, 20, bias=bias))


def test_offsets_past_32_bits(device):
    """C and the 8-bit logits larger than 2^31 elements: the last rows and columns are read and written right."""
    N, D, V = 3, 8192, 270000  # C: 2.2e9 elements
    g = torch.Generator(device=device).manual_seed(19)
    C = torch.empty(V, D, dtype=torch.bfloat16, device=device)
    for i in range(0, V, 30000):
        C[i:i + 30000] = (torch.randn(30000, D, generator=g, device=device) / math.sqrt(D)).bfloat16()
    best = torch.tensor([V - 1, V - 2000, 5], device=device)
    E = (torch.randn(N, D, generator=g, device=device) + 12 * C[best].float()).bfloat16()
    tok = torch.stack((best, torch.tensor([V - 2, 7, 262144], device=device)), 1)
    out = lce.linear_logprobs(E, C, tok, top_k=3)
    z = torch.cat([E.double() @ C[i:i + 30000].double().T for i in range(0, V, 30000)], 1)
    ref = torch.log_softmax(z, 1)
    dz = 2.0 ** -14 * (E.double().abs() @ C[best].double().abs().T).amax(1)
    assert ((out.logprobs.double() - ref.gather(1, tok)).abs() <=
            2 * dz[:, None] + 2.0 ** -18 * (1 + ref.gather(1, tok).abs())).all()
    assert torch.equal(out.top_ids, torch.sort(z, 1, descending=True)[1][:, :3])
    lp, H, lse, *_ = L.cce_logprobs(E, C, tok)
    gl = torch.randn(N, 2, device=device)
    dE, dC, _ = L.cce_logprobs_backward(E, C, tok, lp, lse, H, None, gl, None)
    G = -ref.exp() * gl.double().sum(1, keepdim=True)
    G.scatter_add_(1, tok, gl.double())
    for rows in (tok.reshape(-1), torch.tensor([262143, 262145, V - 1], device=device)):
        want = G[:, rows].T @ E.double()
        assert (dC[rows].double() - want).norm() <= 3 * 2.0 ** -8 * (G[:, rows].abs().T @ E.double().abs()).norm()
    del C, z, ref, dC, G
    # 8-bit logits: 36000 x 65000 = 2.3e9
    N, D, V = 36000, 64, 65000
    c = (torch.randn(V, D, generator=g, device=device) / 8).bfloat16()
    e = torch.randn(N, D, generator=g, device=device).bfloat16()
    q = lce.quantize_int8(c)
    got = lce.int8_linear(e, q)
    for r in (0, 17, N - 1):
        want = lce.int8_linear(e[r:r + 1], q)[0]
        assert torch.equal(got[r], want)
    del got
    torch.cuda.empty_cache()


def test_a_teacher_and_a_student(device):
    """A run of the operators together: a teacher's 8-bit head gives alternatives, the student is pulled towards them
    with an entropy term; the gradient is that of the same loss written out."""
    N, D, V, k = 150, 128, 4000, 6
    E, C, _, _ = make(N, D, V, 20, device)
    Et, Ct, _, _ = make(N, D, V, 21, device)
    teacher = lce.linear_top_logprobs(Et, lce.quantize_int8(Ct), k, temperature=2.0)
    e, c = E.clone().requires_grad_(True), C.clone().requires_grad_(True)
    out = lce.linear_logprobs(e, c, teacher.ids, temperature=2.0)
    weight = teacher.logprobs.exp()
    loss = (weight * (teacher.logprobs - out.logprobs)).sum() - 0.01 * out.entropy.sum()
    loss.backward()
    ref, tol = grad_reference(E, C, None, teacher.ids, 2.0, -weight, torch.full((N,), -0.01, device=device))
    check_grads((e.grad, c.grad), ref, tol)
    # and beside the loss that the framework had: its token losses are the negative log-probabilities
    nll = ops.linear_cross_entropy(E, C, teacher.ids[:, 0], reduction="none")
    lp = lce.linear_logprobs(E, C, teacher.ids[:, 0]).logprobs
    assert (nll + lp).abs().max() <= 2 * logit_tol(E, C).max().item() + 2.0 ** -18 * (1 + lp.abs().max().item())


def scattered_tokens(N, V, gen):
    """32 tokens a position: apart, 20 side by side in every third row, equal ones in the next, one at either end, in
    any order, some asking for nothing, and all of them in row 17."""
    tok = torch.randint(0, V, (N, 32), generator=gen)
    tok[::3, :20] = torch.randint(0, V - 20, (len(tok[::3]), 1), generator=gen) + torch.randperm(20, generator=gen)
    tok[1::3, 5:9] = tok[1::3, 4:5]
    tok[:, 10] = V - 1
    tok[:, 11] = 0
    tok[torch.rand(N, 32, generator=gen) < 0.1] = IGNORE
    tok[17] = IGNORE
    return tok


@pytest.mark.parametrize("N,V", [(700, 80001), (300, 5000), (2100, 131)])
def test_many_tokens_are_met_wherever_they_lie(device, N, V):
    """Each of 32 tokens has the log-probability that it has alone (the same logit, the same sums: to the bit).
    700 x 80001 walks its columns from the middle of a share on and turns round."""
    gen = torch.Generator().manual_seed(N + V)
    E = torch.randn(N, 64, generator=gen).bfloat16().to(device)
    C = torch.randn(V, 64, generator=gen).bfloat16().to(device)
    tok = scattered_tokens(N, V, gen).to(device)
    many = lce.linear_logprobs(E, C, tok)
    for k in range(32):
        alone = lce.linear_logprobs(E, C, tok[:, k])
        assert torch.equal(many.logprobs[:, k], alone.logprobs)
        asks = tok[:, k] != IGNORE
        assert torch.equal(many.entropy[asks], alone.entropy[asks])
    assert many.entropy[17] == 0 and (many.logprobs[17] == 0).all()


@pytest.mark.parametrize("N,V", [(300, 5000), (150, 131)])
def test_gradients_of_many_tokens(device, N, V):
    E, C, bias, _ = make(N, 64, V, 3 * N + V, device, True, 1)
    gen = torch.Generator().manual_seed(V)
    tok = scattered_tokens(N, V, gen).to(device)
    g = torch.randn(N, 32, generator=gen).to(device)
    h = torch.randn(N, generator=gen).to(device)
    lp, H, lse, *_ = L.cce_logprobs(E, C, tok, 0, bias, 0.7)
    out = L.cce_logprobs_backward(E, C, tok, lp, lse, H, None, g, h, bias=bias, temperature=0.7, out_fp32=ops.OUT_FP32)
    ref, tol = grad_reference(E, C, bias, tok, 0.7, g, h)
    check_grads((out[0], out[1], out[3]), ref, tol)
    assert (out[0][17] == 0).all()


def test_many_tokens_of_a_long_batch_with_alternatives(device):
    """Rows are taken a slab at a time there, their tokens too."""
    N, V = 4500, 700
    E, C, _, _ = make(N, 64, V, 29, device, K=1)
    tok = scattered_tokens(N, V, torch.Generator().manual_seed(2)).to(device)
    lp, H, lse, _, tl, ti = L.cce_logprobs(E, C, tok, 3, check=True)
    check_logprobs(E, C, None, tok, 1.0, lp, H)
    check_top(E, C, None, 3, 1.0, lce.TopLogprobs(tl, ti))
    q = lce.quantize_int8(C)
    lp8, H8, *_ = L.cce_logprobs(E, q, tok, 3, check=True)
    alone, Ha, *_ = L.cce_logprobs(E, q, tok, check=True)
    # the same logits (8-bit products are exact); only the order of the statistics' sums differs
    assert ((lp8 - alone).abs() <= 2.0 ** -18 * (1 + alone.abs())).all()
    assert ((H8 - Ha).abs() <= 2.0 ** -18 * (1 + math.log(V))).all()
