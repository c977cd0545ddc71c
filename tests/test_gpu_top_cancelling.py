"""Alternatives where most of what a logit adds up cancels: two large features of opposite sign, a bias that takes the
product away. Neighbours then lie closer than the rounding of their 32-bit sums, which goes by the magnitudes added, and
their order has to come from 64 bits all the same, whatever the batch (up to 128 rows, and above, the candidates' logits
are added up in another order). Every id is compared with the sort of the logits in 64 bits."""
import math

import pytest
import torch

import linear_cross_entropy_06_b200 as lce

from test_gpu_int8_head import logits64 as logits64_int8, rows64
from test_gpu_logprobs import logits64

pytestmark = pytest.mark.gpu

V, k = 20000, 12


def check(E, C, bias, z, counts=(300, 128, 129, 17, 1)):
    want = torch.sort(z, dim=1, descending=True, stable=True)[1][:, :k]
    wrong = {n: (lce.linear_top_logprobs(E[:n], C, k, bias=bias).ids != want[:n]).any(1).sum().item() for n in counts}
    assert not any(wrong.values()), f"rows with other ids, by batch: {wrong}"


@pytest.mark.parametrize("D", [1024, 2304])
@pytest.mark.parametrize("size", [512, 2048])
def test_opposed_features(device, D, size):
    g = torch.Generator().manual_seed(D + size)
    E, C = torch.randn(300, D, generator=g), torch.randn(V, D, generator=g) / math.sqrt(D)
    x = size / 64 * (1 + torch.rand(V, generator=g)).bfloat16().float()
    E[:, 0] = E[:, 700] = 64
    C[:, 0], C[:, 700] = x, -x
    E, C = E.bfloat16().to(device), C.bfloat16().to(device)
    check(E, C, None, logits64(E, C, None))


@pytest.mark.parametrize("int8", [False, True])
def test_a_bias_that_takes_the_product_away(device, int8):
    """Products of about 1000, all but equal: rows of C that differ by a step of bf16 in 8 places, or 8-bit rows that
    differ by 1 in 8 places and whose scales make up for it up to 1e-5."""
    N, D = 300, 512
    g = torch.Generator().manual_seed(3)
    e = torch.randn(D, generator=g)
    E = (e + 0.05 * torch.randn(N, D, generator=g)).bfloat16().to(device)
    C = (1000 / (e * e).sum() * e).bfloat16().expand(V, D).clone()
    at = torch.randint(0, D, (V, 8), generator=g)
    step = torch.randint(-1, 2, (V, 8), generator=g)
    if int8:
        q, s = rows64(C)
        q = q.scatter(1, at, (q.gather(1, at) + step).clamp(-127, 127))
        sums = (q * rows64(E[:1].cpu())[0]).sum(1)
        scale = (s * sums.mean() / sums * (1 + 1e-5 * torch.randn(V, generator=g))).float()
        C = lce.Int8Rows(q.to(torch.int8).to(device), scale.to(device))
    else:
        bits = C.view(torch.int16)
        C = bits.scatter(1, at, bits.gather(1, at) + step.to(torch.int16)).view(torch.bfloat16).to(device)
    bias = torch.full((V,), -1000.0).bfloat16().to(device)
    z = (logits64_int8 if int8 else logits64)(E, C, bias)
    check(E, C, bias, z)
