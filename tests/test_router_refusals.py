"""What moe_linear, moe_linear_grad, moe_route and moe_route_grad refuse.  No
call here reaches a GPU: the device pointers are never dereferenced."""
import pytest
import torch

from moe_prefill_routing_gb300 import binding as B
from moe_prefill_routing_gb300 import build as build_mod

FAKE = 0x10000
BIG = 1 << 40


@pytest.fixture(scope="module")
def lib():
    build_mod.build()
    return B.lib()


def _call(fn, names, base, **kw):
    a = {**base, **kw}
    return fn(*[a[n] for n in names])


LIN = ("x ldx W bias residual ldr dtype act T K N pre y ldy y_dtype status stream").split()
LIN_OK = dict(x=FAKE, ldx=64, W=FAKE, bias=None, residual=None, ldr=0, dtype=0, act=0, T=4, K=64,
              N=10, pre=None, y=FAKE, ldy=10, y_dtype=0, status=None, stream=None)


@pytest.mark.parametrize("kw,rc", [
    (dict(dtype=2), "DTYPE"), (dict(dtype=7), "DTYPE"), (dict(y_dtype=1), "DTYPE"),
    (dict(T=-1), "SHAPE"), (dict(K=0), "SHAPE"), (dict(K=60), "SHAPE"), (dict(N=0), "SHAPE"),
    (dict(act=5), "SHAPE"), (dict(act=-1), "SHAPE"), (dict(ldx=56), "SHAPE"),
    (dict(ldx=68), "SHAPE"), (dict(T=(1 << 31) - 511), "SHAPE"),
    (dict(N=(1 << 31) - 1, ldy=1 << 31), "SHAPE"), (dict(ldy=9), "SHAPE"), (dict(residual=FAKE, ldr=9), "SHAPE"),
    (dict(x=None), "NULL"), (dict(W=None), "NULL"), (dict(y=None), "NULL"),
    (dict(x=FAKE + 8), "ALIGN"), (dict(W=FAKE + 2), "ALIGN"), (dict(y=FAKE + 1), "ALIGN"),
    (dict(y=FAKE + 2, y_dtype=2), "ALIGN"), (dict(bias=FAKE + 2), "ALIGN"),
    (dict(residual=FAKE + 1, ldr=10), "ALIGN"), (dict(pre=FAKE + 1), "ALIGN"),
    (dict(status=FAKE + 2), "ALIGN")])
def test_linear(lib, kw, rc):
    assert _call(lib.moe_linear, LIN, LIN_OK, **kw) == getattr(B, "MOE_ERR_" + rc)


def test_route_needs_a_workspace_for_statistics(lib):
    none = dict(counts=None, prob=None, loss=None)
    for name in none:
        kw = {**none, name: FAKE, "ws": None}
        assert _call(lib.moe_route, ROUTE, ROUTE_OK, **kw) == B.MOE_ERR_NULL
    assert _call(lib.moe_route, ROUTE, ROUTE_OK, **none, ws_bytes=8) == B.MOE_ERR_WORKSPACE


def test_linear_without_tokens_does_nothing(lib):
    assert _call(lib.moe_linear, LIN, LIN_OK, T=0, x=None, y=None) == B.MOE_OK


GRAD = ("x ldx W pre dy lddy dy_dtype dtype act T K N dx dW dw_dtype db ws ws_bytes status "
        "stream").split()
GRAD_OK = dict(x=FAKE, ldx=64, W=FAKE, pre=None, dy=FAKE, lddy=10, dy_dtype=0, dtype=0, act=0, T=4,
               K=64, N=10, dx=FAKE, dW=FAKE, dw_dtype=0, db=FAKE, ws=FAKE, ws_bytes=BIG,
               status=None, stream=None)


@pytest.mark.parametrize("kw,rc", [
    (dict(dtype=2), "DTYPE"), (dict(dy_dtype=1), "DTYPE"), (dict(dw_dtype=1), "DTYPE"),
    (dict(T=-1), "SHAPE"), (dict(K=12), "SHAPE"), (dict(N=0), "SHAPE"), (dict(act=9), "SHAPE"),
    (dict(lddy=9), "SHAPE"), (dict(ldx=63), "SHAPE"), (dict(ws=None), "NULL"),
    (dict(W=None), "NULL"), (dict(x=None), "NULL"), (dict(dy=None), "NULL"),
    (dict(act=2), "NULL"), (dict(ws_bytes=16), "WORKSPACE"), (dict(ws=FAKE + 64), "ALIGN"),
    (dict(dy=FAKE + 1), "ALIGN"), (dict(dW=FAKE + 2, dw_dtype=2), "ALIGN"),
    (dict(db=FAKE + 2), "ALIGN"), (dict(x=FAKE + 4), "ALIGN")])
def test_linear_grad(lib, kw, rc):
    assert _call(lib.moe_linear_grad, GRAD, GRAD_OK, **kw) == getattr(B, "MOE_ERR_" + rc)


def test_linear_grad_workspace(lib):
    # dP in 16 bits with rows of a multiple of 8, and 128 rows of fp32 column sums
    assert B.linear_grad_workspace_bytes(100, 33) >= 100 * 40 * 2 + 128 * 33 * 4
    assert B.linear_grad_workspace_bytes(1 << 20, 1 << 14) >= 1 << 35
    assert B.linear_grad_workspace_bytes(-1, 4) == 0


ROUTE = ("logits ld l_dtype bias mask T E k score norm scale ids w counts prob loss ws ws_bytes "
         "stream").split()
ROUTE_OK = dict(logits=FAKE, ld=16, l_dtype=2, bias=None, mask=None, T=4, E=16, k=2, score=0,
                norm=1, scale=1.0, ids=FAKE, w=FAKE, counts=FAKE, prob=FAKE, loss=FAKE, ws=FAKE,
                ws_bytes=BIG, stream=None)


@pytest.mark.parametrize("kw,rc", [
    (dict(l_dtype=3), "DTYPE"), (dict(T=-1), "SHAPE"), (dict(E=0), "SHAPE"),
    (dict(E=4097, ld=4097), "SHAPE"), (dict(k=0), "SHAPE"), (dict(k=17), "SHAPE"),
    (dict(E=512, ld=512, k=257), "SHAPE"), (dict(ld=15), "SHAPE"), (dict(score=2), "SHAPE"),
    (dict(T=1 << 30, k=2), "SHAPE"), (dict(logits=None), "NULL"), (dict(ids=None), "NULL"),
    (dict(w=None), "NULL"), (dict(ws=None), "NULL"), (dict(ws_bytes=255), "WORKSPACE"),
    (dict(logits=FAKE + 2), "ALIGN"), (dict(logits=FAKE + 1, l_dtype=0), "ALIGN"),
    (dict(ws=FAKE + 128), "ALIGN"), (dict(counts=FAKE + 2), "ALIGN"),
    (dict(bias=FAKE + 1), "ALIGN")])
def test_route(lib, kw, rc):
    assert _call(lib.moe_route, ROUTE, ROUTE_OK, **kw) == getattr(B, "MOE_ERR_" + rc)


RGRAD = ("logits ld l_dtype mask ids counts dw dloss T E k score norm scale dlogits ldd "
         "stream").split()
RGRAD_OK = dict(logits=FAKE, ld=16, l_dtype=2, mask=None, ids=FAKE, counts=FAKE, dw=FAKE,
                dloss=FAKE, T=4, E=16, k=2, score=0, norm=1, scale=1.0, dlogits=FAKE, ldd=16,
                stream=None)


@pytest.mark.parametrize("kw,rc", [
    (dict(l_dtype=-1), "DTYPE"), (dict(E=5000, ld=5000, ldd=5000), "SHAPE"), (dict(k=17), "SHAPE"),
    (dict(ldd=8), "SHAPE"), (dict(score=-1), "SHAPE"), (dict(logits=None), "NULL"),
    (dict(ids=None), "NULL"), (dict(dlogits=None), "NULL"), (dict(dw=FAKE + 2), "ALIGN"),
    (dict(dloss=FAKE + 2), "ALIGN"), (dict(dlogits=FAKE + 2), "ALIGN")])
def test_route_grad(lib, kw, rc):
    assert _call(lib.moe_route_grad, RGRAD, RGRAD_OK, **kw) == getattr(B, "MOE_ERR_" + rc)


def test_route_grad_without_tokens_does_nothing(lib):
    assert _call(lib.moe_route_grad, RGRAD, RGRAD_OK, T=0, logits=None) == B.MOE_OK


def test_binding_refuses_before_the_library():
    x = torch.zeros((4, 64), dtype=torch.bfloat16)
    W = torch.zeros((10, 64), dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        B.linear(x, W)
    with pytest.raises(ValueError, match="dtype"):
        B.linear(x.float(), W)
    with pytest.raises(ValueError, match="expected"):
        B.linear(x, W, y=torch.zeros((4, 10)), out_dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        B.route(torch.zeros((4, 8)), 2)
