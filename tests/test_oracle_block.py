"""The 64-bit definitions of the block norm and of MXFP4 rows on the CPU:
hand-computed values, every gradient against central differences, and the MXFP4
codec against the weights' one."""
import numpy as np
import pytest

import oracle
from oracle import block as D


def test_norm_by_hand():
    x = np.array([[3.0, 4.0]])
    # mean square of (3, 4) is 12.5
    assert np.allclose(D.normed(x, np.array([1.0, 2.0]), eps=0.0),
                       [[3 / 12.5 ** 0.5, 8 / 12.5 ** 0.5]], rtol=1e-15)
    xn = D.stream(x, np.array([[0.0, 2.0]]), post=np.array([1.0, 3.0]), gate=np.array([0.0]),
                  gate_act="sigmoid", alpha=2.0, eps=0.0)
    # o / sqrt(2) = (0, sqrt 2), times 3, times 1/2
    assert np.allclose(xn, [[6.0, 8.0 + 1.5 * 2 ** 0.5]], rtol=1e-15)
    xn = D.stream(x, np.array([[0.0, 2.0]]), post_norm=False, mask=np.array([0]))
    assert np.array_equal(xn, [[0.0, 0.0]])


@pytest.mark.parametrize("post_norm", [True, False])
@pytest.mark.parametrize("gate", [None, "none", "sigmoid"])
@pytest.mark.parametrize("post", [True, False])
def test_gradients_against_differences(post_norm, gate, post):
    rng = np.random.default_rng(5)
    T, d, eps, alpha = 3, 7, 1e-3, 0.7
    mask = np.array([1, 0, 1])
    v = {"x": rng.normal(size=(T, d)), "o": rng.normal(size=(T, d)), "pre": rng.normal(size=d)}
    if post:
        v["post"] = rng.normal(size=d)
    if gate:
        v["gate"] = rng.normal(size=T)
    how = dict(mask=mask, post_norm=post_norm, gate_act=gate or "none", alpha=alpha, eps=eps)
    dxn, dh = rng.normal(size=(T, d)), rng.normal(size=(T, d))

    def total(**kw):
        a = {**v, **kw}
        xn = D.stream(a["x"], a["o"], a.get("post"), a.get("gate"), **how)
        h = D.normed(xn, a["pre"], mask=mask, eps=eps)
        # rows without a mask count for nothing
        return np.sum((dxn * xn + dh * h)[mask == 1])

    xn = D.stream(v["x"], v["o"], v.get("post"), v.get("gate"), **how)
    got, size = D.grads(xn, v["o"], dxn, dh, v["pre"], v.get("post"), v.get("gate"), **how)
    assert set(got) == {"dx", "do", "dpre"} | ({"dpost"} if post else set()) | (
        {"dgate"} if gate else set())
    step = 1e-5
    for name in v:
        want = np.zeros(v[name].shape)
        for i in np.ndindex(v[name].shape):
            e = np.zeros(v[name].shape)
            e[i] = step
            want[i] = (total(**{name: v[name] + e}) - total(**{name: v[name] - e})) / (2 * step)
        g = got["d" + name]
        # a third derivative of at most some tens times step^2 / 6, and rounding
        assert np.max(np.abs(g - want)) < 1e-7, name
        assert np.all(np.abs(g) <= size["d" + name] * (1 + 1e-12))


def test_gradients_without_a_block():
    rng = np.random.default_rng(6)
    xn, dh, pre = rng.normal(size=(2, 5)), rng.normal(size=(2, 5)), rng.normal(size=5)
    got, _ = D.grads(xn, dh=dh, pre=pre)
    step = 1e-5
    for i in np.ndindex(xn.shape):
        e = np.zeros(xn.shape)
        e[i] = step
        want = np.sum(dh * (D.normed(xn + e, pre) - D.normed(xn - e, pre))) / (2 * step)
        assert abs(got["dx"][i] - want) < 1e-8


def test_mx_by_hand():
    v = np.zeros((1, 64))
    v[0, :10] = [4.0, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, -0.1, 7.9]
    v[0, 32] = np.inf
    code, scale = D.mx_encode(v)
    # a block maximum of 7.9 = 1.975 x 4: scale 1; ties to the even code
    assert list(code[0, :10]) == [6, 0, 2, 2, 4, 4, 6, 6, 8, 7]
    assert list(scale[0]) == [127, 255] and not code[0, 32:].any()
    values = D.mx_values(code, scale)
    assert list(values[0, :10]) == [4, 0, 1, 1, 2, 2, 4, 4, 0, 6] and np.isnan(values[0, 32:]).all()


def test_mx_against_the_weights_codec():
    """Blocks along K of weights [1, K, M] hold what rows [M, K] do."""
    rng = np.random.default_rng(7)
    K, M = 96, 20
    w = (rng.normal(size=(K, M)) * np.exp(8 * rng.normal(size=(1, M)))).astype(np.float32)
    bits = (w.view(np.uint32) >> 16).astype(np.uint16)  # bf16 values
    w = (bits.astype(np.uint32) << 16).view(np.float32)
    codes, scales = oracle.quantize_mxfp4(bits[None])
    code, scale = D.mx_encode(w.T)
    assert np.array_equal(scale, scales[0].T)
    # the oracle's weights: two features a byte, the even one in the low half
    assert np.array_equal(code.T[:, 0::2] | code.T[:, 1::2] << 4, codes[0])


def test_mx_layout_round_trip():
    rng = np.random.default_rng(8)
    code = rng.integers(0, 16, size=(150, 160)).astype(np.uint8)
    scale = rng.integers(0, 255, size=(150, 5)).astype(np.uint8)
    codes, tiles = D.mx_pack(code, scale)
    assert codes.shape == (150, 80) and tiles.shape == (2, 2, 512)
    assert codes[3, 4] == code[3, 8] | code[3, 9] << 4
    assert tiles[1, 1, 16 * 5 + 0] == scale[133, 4]  # row 133 is row 5 of its tile
    assert tiles[0, 0, 16 * 7 + 4 * 2 + 3] == scale[71, 3]
    c, s = D.mx_unpack(codes, tiles)
    assert np.array_equal(c, code) and np.array_equal(s, scale)
