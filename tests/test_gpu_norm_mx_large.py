"""Tensors whose elements lie past 2^31: the last rows come out as those rows by
themselves do."""
import pytest
import torch

from moe_prefill_routing_gb300 import binding as B

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
T, D, LAST = 1_100_000, 2048, 300  # 2.25e9 elements


def _big(seed, rows=T, d=D):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.empty(rows, d, dtype=BF, device="cuda")
    for part in x.split(100_000):
        part.normal_(generator=g)
    return x


def test_norm_and_its_gradient():
    x, o = _big(1), _big(2)
    w = torch.linspace(0.5, 1.5, D, device="cuda")
    r = B.block_norm(x, o, pre=w, post=w, mxfp4=True)
    few = B.block_norm(x[-LAST:], o[-LAST:], pre=w, post=w)
    assert torch.equal(r["xn"][-LAST:], few["xn"]) and torch.equal(r["h"][-LAST:], few["h"])
    q = B.quantize_rows_mxfp4(few["h"])
    assert torch.equal(r["mx"].codes[-LAST:], q.codes)
    y = B.dequantize_rows_mxfp4(r["mx"])
    assert torch.equal(y[-LAST:], B.dequantize_rows_mxfp4(q))
    del y
    g = B.block_norm_grad(r["xn"], o, dxn=x, dh=r["h"], pre=w, post=w, weights=False)
    want = B.block_norm_grad(few["xn"], o[-LAST:], dxn=x[-LAST:], dh=few["h"], pre=w, post=w,
                             weights=False)
    assert torch.equal(g["dx"][-LAST:], want["dx"]) and torch.equal(g["do"][-LAST:], want["do"])


def test_rows_to_mxfp4():
    x = _big(3)
    q, few = B.quantize_rows_mxfp4(x), B.quantize_rows_mxfp4(x[-LAST:])
    assert torch.equal(q.codes[-LAST:], few.codes)


@pytest.mark.parametrize("out", [BF, F32])
def test_product(out):
    rows, N = 300_000, 8192  # 2.46e9 outputs
    x = _big(4, rows, 64)
    W = B.quantize_rows_mxfp4(_big(5, N, 64))
    y = B.linear_mxfp4(x, W, out_dtype=out)
    assert torch.equal(y[-LAST:], B.linear_mxfp4(x[-LAST:], W, out_dtype=out))
    assert torch.equal(y[:LAST], B.linear_mxfp4(x[:LAST], W, out_dtype=out))
    keep = y[-LAST:].clone()
    B.linear_mxfp4(x, W, residual=y, y=y)
    assert torch.equal(y[-LAST:], B.linear_mxfp4(x[-LAST:], W, residual=keep, out_dtype=out))
