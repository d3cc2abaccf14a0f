"""Gradients of moe_block_norm where its values are large or small, or a gate
is far from 0.

Bounds as in test_gpu_block_norm.py, of which these are further cases: 2^-16 of the
magnitudes that a value is made of.  Rows are scaled by a power of two that leaves
their squares in fp32's range; with those of 2^58 a gradient of o lies around 2^-116,
whose smallest elements are subnormal: at most eight steps of such an element, each
off by half of 2^-149, 2^-147 in all."""
import numpy as np
import pytest
import torch

from oracle import block as D
from test_gpu_block_norm import BF, F32, HALF, _f64, _inputs, _rand

from moe_prefill_routing_gb300 import binding as B

pytestmark = pytest.mark.gpu


def _within(got, ref, tol, what):
    rel, small = HALF[got.dtype]
    tol = tol + 2.0 ** -147
    err = np.abs(_f64(got) - ref)
    bound = tol + rel * (np.abs(ref) + tol) + small
    assert np.all(err <= bound), (what, float(np.max(err / bound)))


def _check(v, gh, gx=None, **how):
    r = B.block_norm(**v, **how)
    names = ("o", "pre", "post", "gate", "mask")
    got = B.block_norm_grad(r["xn"], dxn=gx, dh=gh, **{n: v[n] for n in names}, **how)
    ref, size = D.grads(_f64(r["xn"]), _f64(v["o"]), _f64(gx), _f64(gh), _f64(v["pre"]),
                        _f64(v["post"]), _f64(v["gate"]), _f64(v["mask"]), **how)
    assert set(got) == set(ref)
    for n in ref:
        assert np.isfinite(ref[n]).all()
        _within(got[n], ref[n], 2.0 ** -16 * size[n], n)


@pytest.mark.parametrize("S,Bt", [(BF, BF), (F32, BF), (F32, F32)])
@pytest.mark.parametrize("exponent", [-47, 44, 50, 58])
@pytest.mark.parametrize("scaled,post_norm", [("x", True), ("o", True), ("xo", True), ("xo", False)])
@pytest.mark.parametrize("d", [100, 2816, 8200])
def test_gradients_of_large_and_small_rows(S, Bt, exponent, scaled, post_norm, d):
    v = _inputs(6, d, S, Bt)
    for n in scaled:
        v[n] = v[n] * 2.0 ** exponent
    _check(v, _rand(91, 6, d).to("cuda", Bt), post_norm=post_norm, alpha=0.5,
           eps=0.0 if exponent < 0 else 1e-6)


@pytest.mark.parametrize("S,Bt", [(BF, BF), (F32, F32)])
@pytest.mark.parametrize("exponent", [-47, 58])
def test_gradients_of_a_norm_alone_of_large_and_small_rows(S, Bt, exponent):
    v = _inputs(6, 1000, S, Bt, o=False)
    v["x"] = v["x"] * 2.0 ** exponent
    _check(v, _rand(91, 6, 1000).to("cuda", Bt), eps=0.0 if exponent < 0 else 1e-6)


def test_gradients_of_large_rows_of_one_sign():
    """Products of a stream and an output around 10^36, thousands of them a row."""
    v = _inputs(4, 2560, F32, F32, gate=False)
    for i, n in enumerate("xo"):
        g = torch.Generator().manual_seed(20 + i)
        v[n] = (2.0 ** 59 * (1 + 3 * torch.rand(4, 2560, generator=g))).cuda()
    _check(v, _rand(91, 4, 2560).cuda(), alpha=1.0)


@pytest.mark.parametrize("S,Bt", [(BF, BF), (F32, F32)])
@pytest.mark.parametrize("d", [64, 2560])
def test_gradient_of_a_sigmoid_far_from_its_middle(S, Bt, d):
    """Its slope is 1/(1 + e^-g) 1/(1 + e^g), each within 2^-21 of itself."""
    at = torch.tensor([-80.0, -30, -17, -9, -4, -1, 0, 1, 4, 9, 17, 30, 80])
    v = _inputs(len(at), d, S, Bt)
    v["gate"] = at.cuda()
    r = B.block_norm(**v, gate_act="sigmoid")
    gx = _rand(92, len(at), d).to("cuda", S)
    how = {n: v[n] for n in ("o", "post", "gate")}
    got = B.block_norm_grad(r["xn"], dxn=gx, gate_act="sigmoid", **how)["dgate"]
    # a plain gate's gradient, times the slope
    ref, size = D.grads(_f64(r["xn"]), _f64(v["o"]), _f64(gx), None, None, _f64(v["post"]),
                        np.ones(len(at)))
    g = at.double().numpy()
    slope = 1 / (1 + np.exp(-g)) / (1 + np.exp(g))
    _within(got, ref["dgate"] * slope, (2.0 ** -16 + 2.0 ** -20) * size["dgate"] * slope, "dgate")
