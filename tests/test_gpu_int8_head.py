"""8-bit rows, the product with them, and the head operators on an 8-bit classifier, on the GPU, against the
definitions in 64 bits.

The integers and scales are exact: q is the integer nearest to x / scale. The integer sums are exact, so a logit
carries the roundings of the fp32 conversion, of scale times scale, of their product and of the bias's addition: under
4 * 2^-24 of |z - bias| plus |z|; bf16 outputs one rounding of 2^-8 more."""
import math

import pytest
import torch

import linear_cross_entropy_06_b200 as lce

from test_gpu_logprobs import IGNORE, check_top, make

pytestmark = pytest.mark.gpu


def rows64(x):
    """(integers, scales fp32) of the rows of x, in 64 bits."""
    scale = (x.double().abs().amax(1) / 127.0).float()  # torch divides fp32 by a number through its reciprocal
    q = torch.where(scale[:, None] > 0, (x.double() / scale.double()[:, None]).round(), 0.0)
    return q, scale


def int8_case(N, D, V, seed, device, bias=False, K=None):
    E, C, b, tok = make(N, D, V, seed, device, bias, K)
    qc, sc = rows64(C)
    return E, lce.Int8Rows(qc.to(torch.int8), sc), b, tok


def logits64(E, C, bias):
    q, s = rows64(E)
    z = (q @ C.values.double().T) * s.double()[:, None] * C.scale.double()
    return z if bias is None else z + bias.double()


def tol32(z, bias):
    part = z if bias is None else z - bias.double()
    return 4 * 2.0 ** -24 * (part.abs() + z.abs()) + 1e-38


@pytest.mark.parametrize("rows,D", [(1, 16), (3, 48), (130, 272), (1000, 4096)])
def test_rows_are_rounded_to_the_nearest_integer(device, rows, D):
    g = torch.Generator().manual_seed(rows + D)
    x = (torch.randn(rows, D, generator=g) * torch.exp(torch.randn(rows, 1, generator=g) * 8)).bfloat16()
    if rows > 2:
        x[0] = 0
        x[1] = torch.arange(D).float() % 255 - 127  # scale 1: every integer, exactly
        x[2] = (torch.arange(D).float() % 254 - 127) / 2  # scale 1/2: halves of it
        x[2, 0] = 63.5
    x = x.to(device)
    out = lce.quantize_int8(x)
    q, s = rows64(x)
    assert torch.equal(out.scale, s)
    assert torch.equal(out.values.double(), q)


def test_halves_go_to_the_even_integer_and_no_quotient_is_rounded_onto_one(device):
    """Rows whose scale makes quotients that are halves, or that fp32 division rounds to one."""
    tops = torch.linspace(1.0, 2.0, 129)[:128].bfloat16().float()
    x = torch.zeros(128, 2048)
    m = (1 + torch.arange(256) / 256).repeat(8)[:2047]
    for i, t in enumerate(tops):
        x[i, 0] = t
        x[i, 1:] = (m * 2.0 ** -(torch.arange(2047) // 256 + 1.0)).clamp(max=float(t))
    x = x.bfloat16().to(device)
    out = lce.quantize_int8(x)
    q, s = rows64(x)
    assert torch.equal(out.scale, s) and torch.equal(out.values.double(), q)


def test_rows_that_are_not_finite_get_the_scale_nan(device):
    x = torch.ones(3, 32, device=device, dtype=torch.bfloat16)
    x[0, 5] = math.inf
    x[1, 31] = math.nan
    out = lce.quantize_int8(x)
    assert torch.isnan(out.scale[:2]).all() and out.scale[2] == torch.tensor(1.0) / 127
    assert (out.values[2] == 127).all()
    C = lce.quantize_int8(torch.randn(100, 32, device=device).bfloat16())
    z = lce.int8_linear(x, C, out_dtype=torch.float32)
    assert torch.isnan(z[:2]).all() and torch.isfinite(z[2]).all()


@pytest.mark.parametrize("N,D,V,bias", [(1, 16, 1, False), (1, 4096, 5000, False), (7, 48, 33, True),
                                        (130, 272, 1001, True), (257, 1040, 50257, False), (1030, 128, 20000, True)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_product(device, N, D, V, bias, dtype):
    E, C, b, _ = int8_case(N, D, V, N + D + V, device, bias)
    got = lce.int8_linear(E, C, bias=b, out_dtype=dtype, check=True)
    z = logits64(E, C, b)
    tol = tol32(z, b)
    if dtype == torch.bfloat16:
        tol = tol + 2.0 ** -8 * (z.abs() + tol)
    assert got.dtype == dtype and got.shape == (N, V)
    worst = ((got.double() - z).abs() / tol).max().item()
    assert worst <= 1.0, worst


@pytest.mark.parametrize("N,D,V,bias,k", [(1, 64, 24, False, 24), (3, 4096, 1000, True, 5), (130, 80, 4099, True, 9),
                                          (700, 256, 20011, False, 20)])
def test_alternatives_on_an_8_bit_head(device, N, D, V, bias, k):
    E, C, b, _ = int8_case(N, D, V, 3 * N + V, device, bias)
    z = logits64(E, C, b)
    check_top(E, None, b, k, 0.8, lce.linear_top_logprobs(E, C, k, bias=b, temperature=0.8), z, tol32(z, b).amax(1))


@pytest.mark.parametrize("N,D,V,bias,K", [(1, 16, 3, False, 1), (129, 272, 1000, True, 3), (600, 128, 40000, False, 1)])
def test_logprobs_on_an_8_bit_head(device, N, D, V, bias, K):
    E, C, b, tok = int8_case(N, D, V, 5 * N + V, device, bias, K)
    out = lce.linear_logprobs(E, C, tok, bias=b, top_k=2)
    z = logits64(E, C, b)
    logp = torch.log_softmax(z, 1)
    wanted = tok != IGNORE
    ref = torch.where(wanted, logp.gather(1, tok.clamp(min=0)), 0.0)
    dz = tol32(z, b).amax(1)
    assert ((out.logprobs.double() - ref).abs() <= 2 * dz[:, None] + 2.0 ** -18 * (1 + ref.abs())).all()
    H = torch.special.entr(logp.exp()).sum(1) * wanted.any(1)
    assert ((out.entropy.double() - H).abs() <= 2 * H * dz + 2.0 ** -18 * (1 + H)).all()
    check_top(E, None, b, 2, 1.0, lce.TopLogprobs(out.top_logprobs, out.top_ids), z, dz)


def test_quantised_head_is_close_to_the_bf16_head(device):
    """The pieces together: quantise a classifier, decode alternatives, score them."""
    E, C, _, _ = make(64, 256, 5000, 77, device)
    q = lce.quantize_int8(C)
    top = lce.linear_top_logprobs(E, q, 4)
    again = lce.linear_logprobs(E, q, top.ids)
    # the same logits, one way through the statistics and one through the sorted lists
    assert (again.logprobs - top.logprobs).abs().max() <= 2.0 ** -18 * 12
    z = lce.int8_linear(E, q, out_dtype=torch.float32)
    assert torch.equal(z.argmax(1), top.ids[:, 0])
