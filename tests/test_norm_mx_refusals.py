"""What moe_block_norm, moe_block_norm_grad and the MXFP4 row calls refuse.  No
call here reaches a GPU: the device pointers are never dereferenced."""
import pytest
import torch

from moe_prefill_routing_gb300 import binding as B
from moe_prefill_routing_gb300 import build as build_mod

FAKE = 0x10000
BIG = 1 << 40
MOST = (1 << 31) - 511


@pytest.fixture(scope="module")
def lib():
    build_mod.build()
    return B.lib()


def _call(fn, names, base, **kw):
    a = {**base, **kw}
    return fn(*[a[n] for n in names])


NORM = ("x ldx x_dtype o ldo b_dtype pre post gate mask T d post_norm gate_act alpha eps xn ldxn "
        "h ldh codes scales stream").split()
NORM_OK = dict(x=FAKE, ldx=64, x_dtype=0, o=FAKE, ldo=64, b_dtype=0, pre=FAKE, post=FAKE, gate=FAKE,
               mask=None, T=4, d=64, post_norm=1, gate_act=0, alpha=1.0, eps=1e-6, xn=FAKE, ldxn=64,
               h=FAKE, ldh=64, codes=FAKE, scales=FAKE, stream=None)
ALONE = dict(o=None, post=None, gate=None, xn=None)


@pytest.mark.parametrize("kw,rc", [
    (dict(x_dtype=3), "DTYPE"), (dict(x_dtype=-1), "DTYPE"), (dict(b_dtype=1), "DTYPE"),
    (dict(b_dtype=2), "DTYPE"), (dict(x_dtype=1, b_dtype=0), "DTYPE"),
    (dict(x_dtype=2, b_dtype=3), "DTYPE"),
    (dict(T=-1), "SHAPE"), (dict(T=MOST), "SHAPE"), (dict(d=0), "SHAPE"),
    (dict(d=16385, ldx=BIG, ldo=BIG, ldxn=BIG, ldh=BIG), "SHAPE"), (dict(ldx=63), "SHAPE"),
    (dict(ldo=63), "SHAPE"), (dict(ldxn=63), "SHAPE"), (dict(ldh=63), "SHAPE"),
    (dict(d=48), "SHAPE"), (dict(gate_act=2), "SHAPE"), (dict(gate_act=-1), "SHAPE"),
    (dict(x=None), "NULL"), (dict(xn=None), "NULL"), (dict(ALONE, pre=None), "NULL"),
    (dict(ALONE, post=FAKE), "NULL"), (dict(ALONE, gate=FAKE), "NULL"), (dict(ALONE, xn=FAKE), "NULL"),
    (dict(codes=None), "NULL"), (dict(scales=None), "NULL"), (dict(pre=None), "NULL"),
    (dict(pre=None, h=None), "NULL"), (dict(h=None, codes=None, scales=None), "NULL"),
    (dict(x=FAKE + 1), "ALIGN"), (dict(o=FAKE + 1), "ALIGN"), (dict(xn=FAKE + 1), "ALIGN"),
    (dict(h=FAKE + 1), "ALIGN"), (dict(pre=FAKE + 2), "ALIGN"), (dict(post=FAKE + 2), "ALIGN"),
    (dict(gate=FAKE + 2), "ALIGN"), (dict(codes=FAKE + 8), "ALIGN"), (dict(scales=FAKE + 8), "ALIGN"),
    (dict(x_dtype=2, x=FAKE + 2), "ALIGN"), (dict(x_dtype=2, xn=FAKE + 2), "ALIGN")])
def test_norm(lib, kw, rc):
    assert _call(lib.moe_block_norm, NORM, NORM_OK, **kw) == getattr(B, "MOE_ERR_" + rc)


def test_norm_without_tokens_does_nothing(lib):
    none = dict(T=0, x=None, o=None, gate=None, xn=None, h=None, codes=None, scales=None)
    assert _call(lib.moe_block_norm, NORM, NORM_OK, **none) == B.MOE_OK
    none = dict(T=0, xn=None, o=None, gate=None, dxn=None, dh=None, dx=None, d_o=None, dgate=None)
    assert _call(lib.moe_block_norm_grad, GRAD, GRAD_OK, **none, dpre=None, dpost=None) == B.MOE_OK
    assert _call(lib.moe_block_norm_grad, GRAD, GRAD_OK, **none, ws=None) == B.MOE_ERR_NULL


GRAD = ("xn ldxn x_dtype o ldo b_dtype pre post gate mask dxn lddxn dh lddh T d post_norm gate_act "
        "alpha eps dx lddx d_o lddo dpre dpost dgate ws ws_bytes stream").split()
GRAD_OK = dict(xn=FAKE, ldxn=64, x_dtype=0, o=FAKE, ldo=64, b_dtype=0, pre=FAKE, post=FAKE, gate=FAKE,
               mask=None, dxn=FAKE, lddxn=64, dh=FAKE, lddh=64, T=4, d=64, post_norm=1, gate_act=1,
               alpha=1.0, eps=1e-6, dx=FAKE, lddx=64, d_o=FAKE, lddo=64, dpre=FAKE, dpost=FAKE,
               dgate=FAKE, ws=FAKE, ws_bytes=BIG, stream=None)


@pytest.mark.parametrize("kw,rc", [
    (dict(b_dtype=1), "DTYPE"), (dict(x_dtype=4), "DTYPE"),
    (dict(T=-1), "SHAPE"), (dict(T=MOST), "SHAPE"), (dict(d=0), "SHAPE"),
    (dict(d=16385, ldxn=BIG, ldo=BIG, lddxn=BIG, lddh=BIG, lddx=BIG, lddo=BIG), "SHAPE"),
    (dict(ldxn=63), "SHAPE"), (dict(ldo=63), "SHAPE"), (dict(lddxn=63), "SHAPE"),
    (dict(lddh=63), "SHAPE"), (dict(lddx=63), "SHAPE"), (dict(lddo=63), "SHAPE"),
    (dict(gate_act=5), "SHAPE"),
    (dict(dx=None), "NULL"), (dict(d_o=None), "NULL"), (dict(xn=None), "NULL"),
    (dict(pre=None), "NULL"), (dict(dxn=None, dh=None), "NULL"), (dict(dh=None), "NULL"),
    (dict(o=None, d_o=None, post=None, gate=None, dpost=None), "NULL"),
    (dict(o=None, d_o=None, post=None, gate=None, dgate=None), "NULL"),
    (dict(gate=None), "NULL"), (dict(ws=None), "NULL"),
    (dict(ws_bytes=4 * 2 * 64 * 4 - 1), "WORKSPACE"),
    (dict(ws=FAKE + 128), "ALIGN"), (dict(xn=FAKE + 1), "ALIGN"), (dict(dxn=FAKE + 1), "ALIGN"),
    (dict(dx=FAKE + 1), "ALIGN"), (dict(o=FAKE + 1), "ALIGN"), (dict(dh=FAKE + 1), "ALIGN"),
    (dict(d_o=FAKE + 1), "ALIGN"), (dict(dpre=FAKE + 2), "ALIGN"), (dict(dpost=FAKE + 2), "ALIGN"),
    (dict(dgate=FAKE + 2), "ALIGN")])
def test_norm_grad(lib, kw, rc):
    assert _call(lib.moe_block_norm_grad, GRAD, GRAD_OK, **kw) == getattr(B, "MOE_ERR_" + rc)


def test_norm_grad_workspace(lib):
    f = lib.moe_block_norm_grad_workspace_bytes
    assert f(4, 64) == 4 * 2 * 64 * 4 and f(-1, 64) == 0 and f(4, 0) == 0 and f(4, 16385) == 0
    assert f(0, 64) == 256 and f(1, 1) == 256
    assert f(1 << 20, 2560) == f(1 << 30, 2560)  # rows of partial sums are bounded


QUANT = "x ldx dtype rows K codes scales stream".split()
QUANT_OK = dict(x=FAKE, ldx=64, dtype=0, rows=4, K=64, codes=FAKE, scales=FAKE, stream=None)


@pytest.mark.parametrize("kw,rc", [
    (dict(dtype=3), "DTYPE"), (dict(rows=-1), "SHAPE"), (dict(rows=MOST), "SHAPE"),
    (dict(K=0), "SHAPE"), (dict(K=48), "SHAPE"), (dict(ldx=63), "SHAPE"), (dict(x=None), "NULL"),
    (dict(codes=None), "NULL"), (dict(scales=None), "NULL"), (dict(x=FAKE + 1), "ALIGN"),
    (dict(x=FAKE + 2, dtype=2), "ALIGN"), (dict(codes=FAKE + 8), "ALIGN"),
    (dict(scales=FAKE + 8), "ALIGN"), (dict(rows=0, x=None, codes=None, scales=None), None)])
def test_rows(lib, kw, rc):
    want = B.MOE_OK if rc is None else getattr(B, "MOE_ERR_" + rc)
    assert _call(lib.moe_quantize_rows_mxfp4, QUANT, QUANT_OK, **kw) == want
    back = "codes scales rows K x ldx dtype stream".split()
    assert _call(lib.moe_dequantize_rows_mxfp4, back, QUANT_OK, **kw) == want


def test_rows_come_back_in_types_that_hold_them(lib):
    back = "codes scales rows K x ldx dtype stream".split()
    assert _call(lib.moe_dequantize_rows_mxfp4, back, QUANT_OK, dtype=1) == B.MOE_ERR_DTYPE


def test_scale_bytes(lib):
    f = lib.moe_mxfp4_scale_bytes
    assert f(1, 32) == 512 and f(128, 128) == 512 and f(129, 160) == 2048
    assert f(0, 32) == 0 and f(-1, 32) == 0 and f(1, 48) == 0
    assert f(1 << 30, 1 << 20) == (1 << 23) * (1 << 13) * 512


LIN = ("x xs W Ws bias residual ldr act T K N y ldy y_dtype status stream").split()
LIN_OK = dict(x=FAKE, xs=FAKE, W=FAKE, Ws=FAKE, bias=None, residual=None, ldr=0, act=0, T=4, K=64,
              N=10, y=FAKE, ldy=10, y_dtype=0, status=None, stream=None)


@pytest.mark.parametrize("kw,rc", [
    (dict(y_dtype=3), "DTYPE"), (dict(y_dtype=-1), "DTYPE"), (dict(T=-1), "SHAPE"),
    (dict(T=MOST), "SHAPE"), (dict(K=0), "SHAPE"), (dict(K=48), "SHAPE"), (dict(N=0), "SHAPE"),
    (dict(N=MOST, ldy=BIG), "SHAPE"), (dict(act=5), "SHAPE"), (dict(act=-1), "SHAPE"),
    (dict(ldy=9), "SHAPE"), (dict(residual=FAKE, ldr=9), "SHAPE"), (dict(x=None), "NULL"),
    (dict(xs=None), "NULL"), (dict(W=None), "NULL"), (dict(Ws=None), "NULL"), (dict(y=None), "NULL"),
    (dict(x=FAKE + 8), "ALIGN"), (dict(xs=FAKE + 8), "ALIGN"), (dict(W=FAKE + 8), "ALIGN"),
    (dict(Ws=FAKE + 8), "ALIGN"), (dict(y=FAKE + 1), "ALIGN"), (dict(y=FAKE + 2, y_dtype=2), "ALIGN"),
    (dict(bias=FAKE + 2), "ALIGN"), (dict(residual=FAKE + 1, ldr=10), "ALIGN"),
    (dict(status=FAKE + 2), "ALIGN"), (dict(T=0, x=None, xs=None, y=None), None)])
def test_linear(lib, kw, rc):
    want = B.MOE_OK if rc is None else getattr(B, "MOE_ERR_" + rc)
    assert _call(lib.moe_linear_mxfp4, LIN, LIN_OK, **kw) == want


ROWS = ("x ldx x_dtype W Ws bias residual ldr act T K N y ldy y_dtype ws ws_bytes status "
        "stream").split()
ROWS_OK = dict(LIN_OK, ldx=64, x_dtype=0, T=20, ws=FAKE, ws_bytes=BIG)


@pytest.mark.parametrize("kw,rc", [
    (dict(y_dtype=3), "DTYPE"), (dict(x_dtype=3), "DTYPE"), (dict(T=-1), "SHAPE"),
    (dict(K=48), "SHAPE"), (dict(N=0), "SHAPE"), (dict(ldx=63), "SHAPE"), (dict(ldy=9), "SHAPE"),
    (dict(x=None), "NULL"), (dict(W=None), "NULL"), (dict(y=None), "NULL"), (dict(ws=None), "NULL"),
    (dict(T=4, x=None, ws=None), "NULL"), (dict(T=4, x=FAKE + 1), "ALIGN"), (dict(T=4, ldx=63), "SHAPE"),
    (dict(ws_bytes=768 + 511), "WORKSPACE"), (dict(ws=FAKE + 128), "ALIGN"),
    (dict(x=FAKE + 1), "ALIGN"), (dict(W=FAKE + 8), "ALIGN"),
    (dict(T=0, x=None, y=None, ws=None, ws_bytes=0), None)])
def test_linear_of_rows(lib, kw, rc):
    want = B.MOE_OK if rc is None else getattr(B, "MOE_ERR_" + rc)
    assert _call(lib.moe_linear_rows_mxfp4, ROWS, ROWS_OK, **kw) == want


def test_linear_of_rows_workspace(lib):
    f = lib.moe_linear_rows_mxfp4_workspace_bytes
    assert f(20, 64, 10) == 768 + 512 and f(0, 64, 10) == 0 and f(20, 48, 10) == 0
    assert f(-1, 64, 10) == 0 and f(20, 64, 0) == 0
    assert f(4, 64, 10) == 0  # quantised by the product's kernel
    assert f(16, 1 << 20, 10) == 16 * (1 << 19) + 8192 * 512  # too long for it
    assert f(1000, 2560, 10) == 1000 * 1280 + 8 * 20 * 512


def test_the_binding_refuses_tensors_that_are_not_on_a_gpu():
    x = torch.zeros(4, 64)
    for call in (lambda: B.block_norm(x, pre=torch.ones(64)), lambda: B.quantize_rows_mxfp4(x),
                 lambda: B.block_norm_grad(x, dh=x, pre=torch.ones(64))):
        with pytest.raises(ValueError, match="CUDA"):
            call()
    with pytest.raises(ValueError, match="multiple of 32"):
        B.Mxfp4Rows.empty(4, 48, "cpu")
