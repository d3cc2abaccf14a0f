"""GELU and its derivative relative to themselves, down to z = -13, where
Phi(z) is 6e-39.  Bound: e^(-z^2/2) from an exponent that was rounded twice,
1.25 * 2^-24 z^2 of itself, and 2^-20 for the rest (a formula good to 8.5e-8,
a reciprocal, an exponential and some ten roundings); 2^-122 where the
exponential leaves fp32's normal numbers; then half a unit of the output."""
import pytest
import torch

from moe_prefill_routing_gb300 import binding as B

pytestmark = pytest.mark.gpu


def _z():
    # every bf16 value of -2^-20 ... -13, and the same of the other sign
    bits = torch.arange(0x3580, 0x4151, dtype=torch.int32)
    z = torch.cat([bits | 0x8000, bits]).to(torch.int16).view(torch.bfloat16)
    return z[:z.numel() // 16 * 16]


def _phi(z):
    z = z.double()
    return 0.5 * torch.special.erfc(-z * 0.5 ** 0.5), torch.exp(-z * z / 2) * 0.3989422804014327


def _rel(z):
    return 2.0 ** -20 + 1.25 * 2.0 ** -24 * z.double() ** 2


@pytest.mark.parametrize("rows", [4, 200])  # few tokens, and pairs of CTAs
@pytest.mark.parametrize("out", [torch.float32, torch.bfloat16])
def test_gelu_tail(rows, out):
    z = _z()
    z = z[:z.numel() // (rows * 16) * rows * 16].reshape(rows, -1).contiguous()
    n = z.shape[1]
    y = B.linear(z.cuda(), torch.eye(n, dtype=torch.bfloat16, device="cuda"), act="gelu",
                 out_dtype=out)
    ref = z.double() * _phi(z)[0]
    tol = _rel(z) * ref.abs() + 2.0 ** -122
    half = torch.finfo(out).eps / 2
    err = (y.cpu().double() - ref).abs()
    bound = tol + half * (ref.abs() + tol) + 2.0 ** -126
    assert bool((err <= bound).all()), float((err / bound).max())


def test_gelu_gradient_tail():
    z = _z()
    n = z.numel()
    x = torch.zeros((1, 8), dtype=torch.bfloat16, device="cuda")
    W = torch.zeros((n, 8), dtype=torch.bfloat16, device="cuda")
    _, _, db = B.linear_grad(x, W, torch.ones((1, n), device="cuda"), pre=z[None].cuda(),
                             act="gelu", need=(False, False, True))
    cdf, pdf = _phi(z)
    want = cdf + z.double() * pdf
    mag = cdf + z.double().abs() * pdf
    err = (db.cpu().double() - want).abs()
    bound = (_rel(z) + 2.0 ** -23) * mag + 2.0 ** -120
    assert bool((err <= bound).all()), float((err / bound).max())
