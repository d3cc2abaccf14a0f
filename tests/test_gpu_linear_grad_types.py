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
    dy32 = dy.dtype == F32
    dx, dW, db = B.linear_grad(x, W, dy, need=need, dw_dtype=dw_dtype)
    xd, Wd, d = x.double(), W.double(), dy.double()
    rel, _ = _half(x.dtype)
    one = 0.0 if dy.dtype == x.dtype else rel
    # fp16: dP scaled to 2^13 at least, subnormals 2^-24 apart
    small = 2.0 ** -38 * float(d.abs().max()) if dy32 and x.dtype == F16 else 0.0
    if need[0]:
        _within(dx, d @ Wd, (one + 2.0 ** -20) * (d.abs() @ Wd.abs()) + small * Wd.abs().sum(0),
                x.dtype)
    if need[1]:
        tol = ((one if piece is None else piece) + 2.0 ** -20) * (d.abs().t() @ xd.abs())
        tol = tol + small * xd.abs().sum(0)
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


@pytest.mark.parametrize("dtype", [BF, F16])
@pytest.mark.parametrize("amp", [1e-9, 1e-3, 1e6])
@pytest.mark.parametrize("T,K,N", [(40, 136, 33), (300, 264, 70), (2000, 520, 515),
                                   (2048, 2560, 512)])
def test_fp32_dy(T, K, N, dtype, amp):
    x = _rand(1, T, K).to(dtype)
    W = _rand(2, N, K, amp=0.05).to(dtype)
    dy = _rand(3, T, N + 1, amp=amp)[:, :N]  # rows without 16-byte alignment
    dy[:, ::3] *= 2.0 ** -12                 # columns of different size
    fits = amp < 1e6 or dtype == BF          # (16-bit outputs of 1e6 do not fit fp16)
    _check(x, W, dy, F32, need=(fits, True, True), piece=2.0 ** -16 if dtype == BF else 2.0 ** -22)
    if fits:
        _check(x, W, dy.contiguous(), dtype)


@pytest.mark.parametrize("dtype", [BF, F16])
def test_fp32_dy_with_an_activation(dtype):
    T, K, N = 257, 264, 136
    x, W = _rand(1, T, K).to(dtype), _rand(2, N, K, amp=0.05).to(dtype)
    dy, pre = _rand(3, T, N, amp=1e-8), _rand(4, T, N, amp=2.0).to(dtype)
    dx, dW, db = B.linear_grad(x, W, dy, pre=pre, act="silu", dw_dtype=F32)
    s = torch.sigmoid(pre.double())
    d = dy.double() * s * (1 + pre.double() * (1 - s))
    xd, Wd = x.double(), W.double()
    # dP in fp32 as in its formula: a few units of 2^-22 of dy max(|pre|, 1)
    fp = 2.0 ** -20 * dy.double().abs() * pre.double().abs().clamp(min=1.0)
    small = 2.0 ** -38 * 4e-8 if dtype == F16 else 0.0
    rel = torch.finfo(dtype).eps / 2
    _within(dx, d @ Wd, (fp + rel * d.abs() + small) @ Wd.abs()
            + 2.0 ** -20 * (d.abs() @ Wd.abs()), dtype)
    two = 2.0 ** -16 if dtype == BF else 2.0 ** -22
    _within(dW, d.t() @ xd, (fp + (two + 2.0 ** -20) * d.abs() + small).t() @ xd.abs(), F32)
    _within(db, d.sum(0), fp.sum(0) + 2.0 ** -20 * d.abs().sum(0), F32)


@pytest.mark.parametrize("dtype", [BF, F16])
@pytest.mark.parametrize("dw_dtype", [F32, None])
def test_fp32_dy_that_is_zero_or_no_number(dtype, dw_dtype):
    T, K, N = 300, 136, 70
    x, W = _rand(1, T, K).to(dtype), _rand(2, N, K).to(dtype)
    dy = _rand(3, T, N, amp=1e-6)
    for g in B.linear_grad(x, W, torch.zeros_like(dy), dw_dtype=dw_dtype):
        assert bool((g == 0).all())
    clean = B.linear_grad(x, W, dy, dw_dtype=dw_dtype)
    dy[7, 5], dy[9, 6] = float("inf"), float("nan")
    dx, dW, db = B.linear_grad(x, W, dy, dw_dtype=dw_dtype)
    rows = [t for t in range(T) if t not in (7, 9)]
    cols = [n for n in range(N) if n not in (5, 6)]
    assert torch.equal(dx[rows], clean[0][rows]) and torch.equal(dW[cols], clean[1][cols])
    assert torch.equal(db[cols], clean[2][cols])
    assert not bool(dx[7].isfinite().any()) and bool(dx[9].isnan().all())
    assert not bool(dW[5].isfinite().any()) and bool(dW[6].isnan().all())


def test_workspace_by_type():
    full = B.linear_grad_workspace_bytes(1000, 300)
    half = B.linear_grad_workspace_bytes(1000, 300, BF, F32)
    assert full - half >= 1000 * 304 * 2 and half < full
    x, W = _rand(1, 1000, 64).to(BF), _rand(2, 300, 64).to(BF)
    dy = _rand(3, 1000, 300)
    ws = torch.empty(half, dtype=torch.uint8, device="cuda")
    B.linear_grad(x, W, dy, ws=ws)
    B.linear_grad(x, W, dy.to(BF), dw_dtype=F32, ws=ws)
    with pytest.raises(B.MoeError) as e:
        B.linear_grad(x, W, dy, dw_dtype=F32, ws=ws)
    assert e.value.code == B.MOE_ERR_WORKSPACE
