"""The 64-bit definitions of the router and the dense projections on the CPU:
hand-computed values, and every gradient against central differences."""
import math

import numpy as np
import pytest

from oracle import router as R

ACTS = ["none", "relu", "silu", "gelu", "gelu_tanh"]


@pytest.mark.parametrize("name", ACTS)
def test_activation_gradient_against_differences(name):
    z = np.array([-6.0, -2.5, -1.0, -0.3, 0.2, 0.7, 1.9, 5.0])
    h = 1e-5
    d = (R.act(z + h, name) - R.act(z - h, name)) / (2 * h)
    # central differences: h^2/6 times a third derivative of at most a few, and eps/h
    assert np.max(np.abs(R.act_grad(z, name) - d)) < 1e-8


def test_activation_values():
    assert R.act(np.array([1.0]), "silu")[0] == pytest.approx(1 / (1 + math.exp(-1)), abs=1e-15)
    assert R.act(np.array([1.0]), "gelu")[0] == pytest.approx(0.8413447460685429, abs=1e-14)
    assert R.act(np.array([1.0]), "gelu_tanh")[0] == pytest.approx(0.8411919906082768, abs=1e-12)
    assert list(R.act(np.array([-2.0, 0.0, 3.0]), "relu")) == [0.0, 0.0, 3.0]


@pytest.mark.parametrize("name", ACTS)
def test_linear_gradients_against_differences(name):
    rng = np.random.default_rng(3)
    T, K, N = 4, 8, 5
    x, W, b = rng.standard_normal((T, K)), rng.standard_normal((N, K)), rng.standard_normal(N)
    dy = rng.standard_normal((T, N))
    _, pre = R.linear(x, W, b, None, name)
    assert np.min(np.abs(pre)) > 1e-3  # no kink of relu within a step
    dx, dW, db = R.linear_grad(x, W, dy, pre, name)

    def value():
        return float((R.linear(x, W, b, None, name)[0] * dy).sum())

    h = 1e-6
    for t, g in ((x, dx), (W, dW), (b, db)):
        for i in np.ndindex(t.shape):
            keep = t[i]
            t[i] = keep + h
            up = value()
            t[i] = keep - h
            down = value()
            t[i] = keep
            assert abs((up - down) / (2 * h) - g[i]) < 1e-6 * (1 + abs(g[i]))


def test_route_worked_example():
    l = np.log(np.array([[1.0, 2.0, 3.0, 4.0], [4.0, 4.0, 1.0, 1.0]]))
    r = R.route(l, 2)
    assert r["ids"].tolist() == [[3, 2], [0, 1]]  # the tie goes to the lower id
    assert np.allclose(r["w"], [[4 / 7, 3 / 7], [0.5, 0.5]], atol=1e-15)
    assert r["counts"].tolist() == [1, 1, 1, 1, 2]
    assert np.allclose(r["prob"], [0.25, 0.3, 0.2, 0.25], atol=1e-15)
    # f_e = 1/4: the balance loss is sum prob = 1, z = log(10)^2
    assert np.allclose(r["loss"], [1.0, math.log(10.0) ** 2], atol=1e-14)


def test_route_closed_masked_and_biased():
    inf = np.inf
    l = np.array([[1.0, -inf, 0.0], [-inf, -inf, -inf], [np.nan, 2.0, inf], [5.0, 5.0, 5.0]])
    r = R.route(l, 2, mask=np.array([1, 1, 1, 0]))
    assert r["ids"].tolist() == [[0, 2], [-1, -1], [1, -1], [-1, -1]]
    assert r["counts"].tolist() == [1, 1, 1, 2]
    assert np.all(r["w"][1] == 0) and r["w"][2].tolist() == [1.0, 0.0]
    b = R.route(l[:1], 1, bias=np.array([-5.0, 9.0, 0.0]), score="sigmoid", norm=False, scale=2.0)
    assert b["ids"].tolist() == [[2]] and b["w"][0, 0] == 1.0  # 2 sigmoid(0), without the bias


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("norm", [True, False])
def test_route_gradient_against_differences(score, norm):
    rng = np.random.default_rng(7)
    T, E, k = 5, 6, 3
    l = 2 * rng.standard_normal((T, E))
    l[1, 2] = -np.inf
    l[2] = np.nan
    mask = np.array([1, 1, 0, 1, 1])
    kw = dict(mask=mask, score=score, norm=norm, scale=1.7)
    r = R.route(l, k, bias=0.3 * rng.standard_normal(E), **kw)
    r["ids"][3, 1] = -1  # an unused slot
    dw, dloss = rng.standard_normal((T, k)), np.array([0.8, -0.3])
    g = R.route_grad(l, r["ids"], r["counts"], dw, dloss, **kw)
    h = 1e-6
    for i in np.ndindex(T, E):
        if not np.isfinite(l[i]):
            assert g[i] == 0.0
            continue
        keep = l[i]
        l[i] = keep + h
        up = R.route_value(l, r["ids"], r["counts"], dw, dloss, **kw)
        l[i] = keep - h
        down = R.route_value(l, r["ids"], r["counts"], dw, dloss, **kw)
        l[i] = keep
        assert abs((up - down) / (2 * h) - g[i]) < 1e-7
