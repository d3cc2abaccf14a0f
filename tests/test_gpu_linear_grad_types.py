"""moe_linear_grad's types against 64-bit products (on the GPU): fp32 dW at
sizes of use, fp32 dy with either operand type, and long reductions.

Bounds.  Half a unit of a type is torch.finfo's eps / 2 (or, for subnormals,
half their spacing).  dP rounded once to the operands' type is off by half a
unit; in two pieces by the square of it.  Sums of R products in fp32 lose
less than 2^-20 of the magnitudes' sum (R up to 16384), in chains or not."""
import pytest
import torch

from moe_prefill_routing_gb300 import binding as B

pytestmark = pytest.mark.gpu

BF, F16, F32 = torch.bfloat16, torch.float16, torch.float32


def _rand(seed, *shape, amp=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return amp * torch.randn(*shape, generator=g, device="cuda")


def _half(dtype):
    f = torch.finfo(dtype)
    return f.eps / 2, f.smallest_normal * f.eps / 2


def _within(got, ref, tol, dtype):
    rel, small = _half(dtype)
    err = (got.double() - ref).abs()
    bound = tol + rel * (ref.abs() + tol) + small
    assert bool((err <= bound).all()), float((err / bound).max())


def _check(x, W, dy, dw_dtype, need=(True, True, True), piece=None):
    """act none; `piece`: the relative error of one value of dP in dW."""
    dx, dW, db = B.linear_grad(x, W, dy, need=need, dw_dtype=dw_dtype)
    xd, Wd, d = x.double(), W.double(), dy.double()
    rel, small = _half(x.dtype)
    one = 0.0 if dy.dtype == x.dtype else rel
    if need[0]:
        _within(dx, d @ Wd, (one + 2.0 ** -20) * (d.abs() @ Wd.abs())
                + (small * Wd.abs().sum(0) if one else 0.0), x.dtype)
    if need[1]:
        tol = ((one if piece is None else piece) + 2.0 ** -20) * (d.abs().t() @ xd.abs())
        _within(dW, d.t() @ xd, tol, dw_dtype)
    if need[2]:
        _within(db, d.sum(0), 2.0 ** -20 * d.abs().sum(0), F32)


@pytest.mark.parametrize("T,K,N", [(2048, 2560, 512), (1024, 2560, 256), (512, 5120, 512),
                                   (1089, 3032, 875), (21, 912, 7602), (4096, 2560, 1024)])
def test_fp32_dw_at_sizes_of_use(T, K, N):
    x, W = _rand(1, T, K).to(BF), _rand(2, N, K, amp=0.05).to(BF)
    dy = _rand(3, T, N, amp=1e-2)
    _check(x, W, dy, F32)
    _check(x, W, dy.to(BF), F32)
    _check(x, W, dy, F32, need=(False, True, False))
