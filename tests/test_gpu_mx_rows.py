"""Rows to MXFP4 and back: codes, scales and values exactly those of the 64-bit
definition (a quantisation decides nothing that 32 bits do not hold exactly)."""
import numpy as np
import pytest
import torch

from oracle import block as D

from moe_prefill_routing_gb300 import binding as B

pytestmark = pytest.mark.gpu

BF, F16, F32 = torch.bfloat16, torch.float16, torch.float32


def _rows(seed, R, K, dtype, spread=3.0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(R, K, generator=g) * torch.exp(spread * torch.randn(R, K // 32, generator=g)
                                                   ).repeat_interleave(32, 1)
    return x.to("cuda", dtype)


def _check(x, q=None):
    q = B.quantize_rows_mxfp4(x) if q is None else q
    code, scale = D.mx_encode(x.double().cpu().numpy())
    codes, tiles = D.mx_pack(code, scale)
    assert np.array_equal(q.codes.cpu().numpy(), codes)
    assert np.array_equal(q.scales.cpu().numpy(), tiles)
    want = D.mx_values(code, scale)
    for dtype in (BF, F32):
        y = B.dequantize_rows_mxfp4(q, dtype)
        assert y.dtype == dtype
        assert np.array_equal(y.double().cpu().numpy(), want, equal_nan=True)
    return q


@pytest.mark.parametrize("R,K", [(1, 32), (1, 64), (2, 96), (31, 128), (33, 160), (128, 256),
                                 (129, 288), (777, 1056), (300, 2560), (5, 11264), (2000, 96)])
@pytest.mark.parametrize("dtype", [BF, F16, F32])
def test_shapes(R, K, dtype):
    _check(_rows(R + K, R, K, dtype))


@pytest.mark.parametrize("dtype", [BF, F16, F32])
@pytest.mark.parametrize("pad", [1, 3, 8, 24])
def test_rows_of_a_wider_tensor(dtype, pad):
    w = torch.full((70, 320 + pad), float("nan"), dtype=dtype, device="cuda")
    w[:, :320] = _rows(3, 70, 320, dtype)
    q = _check(w[:, :320])
    y = torch.full((70, 320 + pad), 5.0, dtype=BF, device="cuda")
    B.dequantize_rows_mxfp4(q, y=y[:, :320])
    # (a NaN, of a half precision infinity's block, is one on both sides)
    want = B.dequantize_rows_mxfp4(q)
    assert torch.equal(y[:, :320].nan_to_num(-1.0), want.nan_to_num(-1.0))
    assert torch.equal(y[:, :320].isnan(), want.isnan()) and (y[:, 320:] == 5).all()


@pytest.mark.parametrize("dtype", [BF, F16, F32])
def test_rows_that_start_anywhere(dtype):
    w = _rows(3, 70, 352, dtype, spread=1.0)
    for at in (1, 2, 5):
        q = _check(w[:, at:at + 320])
        y = torch.full((70, 352), 5.0, dtype=F32, device="cuda")
        B.dequantize_rows_mxfp4(q, y=y[:, at:at + 320])
        assert torch.equal(y[:, at:at + 320], B.dequantize_rows_mxfp4(q, F32))
        assert (y[:, :at] == 5).all() and (y[:, at + 320:] == 5).all()


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("R,K", [(1, 32), (5, 96), (130, 160), (33, 2816), (700, 4128)])
def test_read_back_at_any_offset(R, K, dtype):
    q = _check(_rows(4, R, K, BF, spread=1.0))
    want = B.dequantize_rows_mxfp4(q, dtype)
    for at, pad in ((1, 0), (0, 1), (3, 4), (2, 0)):
        big = torch.full((R * (K + pad) + 16,), 5.0, dtype=dtype, device="cuda")
        y = big[at:at + R * (K + pad)].view(R, K + pad)[:, :K]
        B.dequantize_rows_mxfp4(q, y=y)
        assert torch.equal(y, want)
        y.fill_(5.0)
        assert (big == 5).all()


def test_every_tie_and_its_neighbours():
    points = torch.tensor([0.0, 0.25, 0.5, 0.75, 1.0, 1.25, 1.5, 1.75, 2.0, 2.5, 3.0, 3.5, 4.0, 5.0,
                           6.0, 7.0])
    v = []
    for p in points:
        for e in (-1, 0, 1):
            b = torch.tensor([p.item()], dtype=F32).view(torch.int32) + e
            v += [b.view(F32).item() if b >= 0 else 0.0]
    v = torch.tensor(v)
    v = torch.cat((v, -v))
    rows = torch.zeros(len(v), 32)
    rows[:, 0] = 7.5  # scale 1
    rows[:, 1] = v
    for k in (-126, -20, 0, 20, 120):
        _check((rows * 2.0 ** k).cuda())


def test_every_exponent():
    e = torch.arange(-149, 128, dtype=torch.float64)
    rows = (1.75 * 2.0 ** e)[:, None] * torch.tensor([1.0, -0.5, 0.3, 0.01] * 8, dtype=torch.float64)
    rows[:, 5] = 0
    _check(rows.to("cuda", F32))
    _check(rows.to("cuda", BF))


def test_zeros_signs_nan_and_infinities():
    x = _rows(4, 6, 128, F32)
    x[0] = 0.0
    x[1] = -0.0
    x[2, 40] = float("nan")
    x[3, 70] = float("inf")
    x[4, 100] = -float("inf")
    for dtype in (BF, F16, F32):
        q = _check(x.to(dtype))
        y = B.dequantize_rows_mxfp4(q)
        assert torch.isnan(y[2, 32:64]).all() and torch.isnan(y).sum() == 96
        assert torch.signbit(y[1]).all() and not torch.signbit(y[0]).any()


def test_given_outputs_and_no_rows():
    x = _rows(9, 40, 224, BF)
    out = B.Mxfp4Rows.empty(40, 224, "cuda")
    out.scales.fill_(99)
    assert B.quantize_rows_mxfp4(x, out) is out
    _check(x, out)  # scale bytes past the last row and block are 0
    q = B.quantize_rows_mxfp4(x[:0])
    assert q.shape == (0, 224) and B.dequantize_rows_mxfp4(q).shape == (0, 224)


def test_refusals():
    x = _rows(9, 40, 224, BF)
    q = B.quantize_rows_mxfp4(x)
    with pytest.raises(ValueError):
        B.quantize_rows_mxfp4(x[:, :48])
    with pytest.raises(ValueError):
        B.quantize_rows_mxfp4(x.double())
    with pytest.raises(ValueError):
        B.quantize_rows_mxfp4(x, B.Mxfp4Rows.empty(41, 224, "cuda"))
    with pytest.raises(ValueError):
        B.dequantize_rows_mxfp4(q, F16)
    with pytest.raises(ValueError):
        B.dequantize_rows_mxfp4(B.Mxfp4Rows(q.codes, q.scales[:, :1].contiguous()))
    with pytest.raises(ValueError):
        B.dequantize_rows_mxfp4(B.Mxfp4Rows(q.codes.cpu(), q.scales))
