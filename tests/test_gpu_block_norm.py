"""moe_block_norm and moe_block_norm_grad against the 64-bit definitions.

Bounds, element by element.  A mean of d squares is a sum of positive numbers,
off by at most (chain + 1) 2^-24 of itself, the chain being 32 products of a
thread, 5 shuffles and 16 warps: 2^-18; half of that reaches its root, and the
root, the reciprocal and the products add a few 2^-23.  Norms are held to 2^-18
of themselves, a row's gradients, which use two sums each of terms of either sign,
to 2^-16 of the magnitudes they are made of.  Sums over rows add at most some 200
numbers in turn (rows of a CTA, CTAs of a warp, warps): 200 2^-24 < 2^-16 of
the magnitudes.  The sigmoid is within 2^-21 of itself.  The output's type adds
half a unit, as in the other tests: torch.finfo's eps / 2, or half the spacing
of subnormals.  h and the gradients are of the stream as it was stored, so the
kernel's own xn is what the definition is given for them."""
import numpy as np
import pytest
import torch

from oracle import block as D

from moe_prefill_routing_gb300 import binding as B

pytestmark = pytest.mark.gpu

BF, F16, F32 = torch.bfloat16, torch.float16, torch.float32
TYPES = [(BF, BF), (F16, F16), (F32, BF), (F32, F16), (F32, F32)]
HALF = {t: (torch.finfo(t).eps / 2, torch.finfo(t).smallest_normal * torch.finfo(t).eps / 2)
        for t in (BF, F16, F32)}


def _rand(seed, *shape, amp=1.0):
    g = torch.Generator().manual_seed(seed)
    return amp * torch.randn(*shape, generator=g)


def _wide(t, pad, dtype):
    """t on the GPU as the first columns of a wider tensor."""
    if not pad:
        return t.to("cuda", dtype)
    w = torch.full((t.shape[0], t.shape[1] + pad), float("nan"), dtype=dtype, device="cuda")
    w[:, :t.shape[1]] = t.to("cuda", dtype)
    return w[:, :t.shape[1]]


def _f64(t):
    return None if t is None else t.detach().double().cpu().numpy()


def _within(got, ref, tol, what=""):
    rel, small = HALF[got.dtype]
    err = np.abs(_f64(got) - ref)
    bound = tol + rel * (np.abs(ref) + tol) + small
    assert np.all(err <= bound), (what, float(np.max(err / bound)))


def _inputs(T, d, S, Bt, o=True, pre=True, post=True, gate=True, mask=False, pad=0, seed=0):
    v = {"x": _wide(_rand(seed, T, d, amp=2.0), pad, S), "o": None, "pre": None, "post": None,
         "gate": None, "mask": None}
    if o:
        v["o"] = _wide(_rand(seed + 1, T, d, amp=0.5), pad, Bt)
        v["post"] = (0.5 + _rand(seed + 2, d, amp=0.2)).cuda() if post else None
        v["gate"] = _rand(seed + 3, T).cuda() if gate else None
    v["pre"] = (1 + _rand(seed + 4, d, amp=0.2)).cuda() if pre else None
    if mask:
        v["mask"] = (torch.arange(T) % 3 != 1).cuda()
        v["x"][~v["mask"]] = float("nan")
        if o:
            v["o"][~v["mask"]] = float("inf")
    return v


def _check(v, post_norm=True, gate_act="none", alpha=1.0, eps=1e-6, mxfp4=False, **kw):
    S = v["x"].dtype
    r = B.block_norm(**v, post_norm=post_norm, gate_act=gate_act, alpha=alpha, eps=eps,
                     mxfp4=mxfp4, **kw)
    m = _f64(v["mask"])
    xn = r["xn"]
    if v["o"] is not None:
        how = dict(mask=m, post_norm=post_norm, gate_act=gate_act, alpha=alpha, eps=eps)
        x, o = _f64(v["x"]), _f64(v["o"])
        ref = D.stream(x, o, _f64(v["post"]), _f64(v["gate"]), **how)
        added = np.abs(ref - D.stream(x, np.zeros_like(o), **how))
        live = np.ones(len(x), bool) if m is None else m.astype(bool)
        size = np.where(live[:, None], np.abs(x), 0) * abs(alpha)
        _within(xn, ref, 2.0 ** -18 * added + 2.0 ** -22 * (size + added), "xn")
        assert xn.dtype == S
    else:
        assert xn is v["x"]
    if v["pre"] is not None:
        h = r["h"]
        ref = D.normed(_f64(xn), _f64(v["pre"]), mask=m, eps=eps)
        _within(h, ref, 2.0 ** -18 * np.abs(ref), "h")
    if mxfp4:
        code, scale = D.mx_encode(_f64(h))
        codes, tiles = D.mx_pack(code, scale)
        assert np.array_equal(r["mx"].codes.cpu().numpy(), codes)
        assert np.array_equal(r["mx"].scales.cpu().numpy(), tiles)
    return r


@pytest.mark.parametrize("d", [1, 2, 7, 8, 9, 31, 32, 64, 100, 255, 256, 257, 1000, 1024, 2560, 2816,
                               4096, 4104, 5120, 8191, 8192, 8200, 11264, 16384])
def test_widths(d):
    _check(_inputs(5, d, BF, BF), gate_act="sigmoid", alpha=0.5)


@pytest.mark.parametrize("S,Bt", TYPES)
@pytest.mark.parametrize("d", [96, 1001, 4608, 9000])
def test_types(S, Bt, d):
    _check(_inputs(9, d, S, Bt, pad=8), alpha=0.7)
    _check(_inputs(9, d, S, Bt, o=False), h_dtype=Bt)


@pytest.mark.parametrize("T", [1, 2, 3, 33, 127, 129, 1000, 5000])
def test_lengths(T):
    _check(_inputs(T, 320, BF, BF, mask=True), mxfp4=True)


@pytest.mark.parametrize("post_norm", [True, False])
@pytest.mark.parametrize("post", [True, False])
@pytest.mark.parametrize("gate", [None, "none", "sigmoid"])
@pytest.mark.parametrize("pre", [True, False])
def test_choices(post_norm, post, gate, pre):
    v = _inputs(40, 264, F16, F16, pre=pre, post=post, gate=gate is not None, mask=True, pad=3)
    _check(v, post_norm=post_norm, gate_act=gate or "none", alpha=1.5, eps=1e-5)


@pytest.mark.parametrize("d", [32, 96, 128, 160, 2560, 4096, 4128, 8224, 16384])
@pytest.mark.parametrize("S,Bt", [(BF, BF), (F32, F32), (F32, F16)])
def test_mxfp4_rows_of_h(d, S, Bt):
    _check(_inputs(130, d, S, Bt), mxfp4=True)
    _check(_inputs(7, d, S, Bt, o=False, mask=True), mxfp4=True, h_dtype=Bt)


@pytest.mark.parametrize("S,Bt", TYPES)
@pytest.mark.parametrize("T,d", [(50, 96), (50, 416), (200, 2592), (3, 8224)])
def test_mxfp4_rows_of_h_from_unaligned_rows(T, d, S, Bt):
    _check(_inputs(T, d, S, Bt, mask=True, pad=3), gate_act="sigmoid", alpha=0.5, mxfp4=True)
    v = _inputs(T, d, S, Bt, o=False, pad=1)
    _check(v, mxfp4=True)


def test_in_place_on_unaligned_rows():
    for S, T, d in ((BF, 400, 263), (F32, 300, 1001), (F16, 50, 99)):
        v = _inputs(T, d, S, S, mask=True, gate=False, pad=2)
        want = _check(v)
        gx, gh = _wide(_rand(5, T, d), 1, S), _wide(_rand(6, T, d), 4, S)
        how = {n: v[n] for n in ("pre", "post", "mask")}
        ref = B.block_norm_grad(want["xn"], v["o"], dxn=gx, dh=gh, **how)
        x, o = v["x"].clone(), v["o"].clone()
        r = B.block_norm(**{**v, "x": x}, xn=x)
        assert r["xn"] is x and torch.equal(x, want["xn"]) and torch.equal(r["h"], want["h"])
        got = B.block_norm_grad(want["xn"], o, dxn=gx, dh=gh, **how, dx=gx, do=o)
        for n in ref:
            assert torch.equal(got[n], ref[n]), n


def test_rows_of_zeros_and_of_one_value():
    v = _inputs(6, 512, BF, BF)
    v["x"][0] = 0
    v["o"][0] = 0
    v["o"][1] = 0
    v["x"][2, 1:] = 0
    v["x"][3] = 2.0 ** 60
    v["x"][4] = 2.0 ** -70
    v["o"][4] = 2.0 ** -70
    r = _check(v, mxfp4=True)
    assert not r["h"][0].any() and torch.isfinite(r["h"]).all()


def test_rows_with_a_nan_or_an_infinity_stay_alone():
    v = _inputs(6, 512, BF, BF)
    clean = _check(v)
    v["x"][1, 5] = float("nan")
    v["o"][3, 7] = float("inf")
    r = B.block_norm(**v, mxfp4=True)
    for name in ("xn", "h"):
        for t in (0, 2, 4, 5):
            assert torch.equal(r[name][t], clean[name][t])
    assert torch.isnan(r["h"][1]).all() and torch.isnan(r["xn"][1]).sum() == 1
    values = B.dequantize_rows_mxfp4(r["mx"])
    assert torch.isnan(values[1]).all() and torch.isfinite(values[0]).all()


def test_in_place_and_rows_left_alone():
    v = _inputs(50, 640, BF, BF, mask=True, gate=False)
    want = _check(v)
    big = torch.full((60, 648), 7.0, dtype=BF, device="cuda")
    x = big[:50, :640]
    x.copy_(v["x"])
    h = torch.full((60, 640), 7.0, dtype=BF, device="cuda")
    r = B.block_norm(**{**v, "x": x}, xn=x, h=h[:50])
    assert r["xn"] is x and torch.equal(x, want["xn"]) and torch.equal(h[:50], want["h"])
    assert (h[50:] == 7).all() and (big[50:] == 7).all() and (big[:, 640:] == 7).all()


@pytest.mark.parametrize("S,Bt", [(BF, BF), (F32, BF), (F32, F32)])
@pytest.mark.parametrize("d", [40, 520, 9000])
def test_rows_that_start_anywhere(S, Bt, d):
    v = _inputs(20, d, S, Bt)
    how = {n: v[n] for n in ("pre", "post", "gate")}
    want = B.block_norm(v["x"], v["o"], **how)
    gx, gh = _rand(7, 20, d).to("cuda", S), _rand(8, 20, d).to("cuda", Bt)
    grads = B.block_norm_grad(want["xn"], v["o"], dxn=gx, dh=gh, **how)
    moved = lambda t, at: torch.cat((torch.full((20, at), 3.0, dtype=t.dtype, device="cuda"), t),  # noqa: E731
                                    1)[:, at:]
    for at in (1, 3):
        x, o = moved(v["x"], at), moved(v["o"], at)
        xn, h = moved(torch.zeros_like(x), at), moved(torch.zeros_like(o), at)
        B.block_norm(x, o, **how, xn=xn, h=h)
        # (sums in another order: 2^-18 of the norm and a rounding to either side)
        for a, b in ((xn, want["xn"]), (h, want["h"])):
            assert torch.allclose(a.float(), b.float(), rtol=2.0 ** -17 + torch.finfo(a.dtype).eps,
                                  atol=2.0 ** -17)
        dx, do = moved(torch.zeros_like(x), at), moved(torch.zeros_like(o), at)
        got = B.block_norm_grad(moved(want["xn"], at), o, dxn=moved(gx, at), dh=moved(gh, at), **how,
                                dx=dx, do=do)
        ref, size = D.grads(_f64(want["xn"]), _f64(v["o"]), _f64(gx), _f64(gh), _f64(v["pre"]),
                            _f64(v["post"]), _f64(v["gate"]))
        for n in ref:
            _within(got[n], ref[n], 2.0 ** -16 * size[n], n)
            _within(grads[n], ref[n], 2.0 ** -16 * size[n], n)
        for t in (xn, h, dx, do):
            assert (t._base[:, :at] == 3).all()


@pytest.mark.parametrize("S,Bt", TYPES)
@pytest.mark.parametrize("T,d", [(40, 1), (40, 3), (33, 5), (20, 13), (9, 255), (200, 263), (7, 1030),
                                 (300, 2815), (3, 4097)])
def test_rows_without_a_gap_at_any_offset(S, Bt, T, d):
    """Rows of odd length one behind the other, in the middle of memory that holds NaN, at every
    element's offset into 16 bytes: a value from beside a row would show."""
    def at(t, i):
        big = torch.full((T * d + 40,), float("nan"), dtype=t.dtype, device="cuda")
        v = big[8 + i:8 + i + T * d].view(T, d)
        v.copy_(t)
        return v

    v = _inputs(T, d, S, Bt, mask=T > 30)
    rest = {n: v[n] for n in ("pre", "post", "gate", "mask")}
    gx, gh = _rand(7, T, d).to("cuda", S), _rand(8, T, d).to("cuda", Bt)
    for i in range(16 // torch.finfo(Bt).bits * 8 if d < 300 else 1, 0, -1):
        j, k = (3 * i) % 8, (5 * i + 1) % 8
        x, o, xn, h = at(v["x"], i), at(v["o"], j), at(v["x"], k), at(v["o"], i)
        r = _check({**rest, "x": x, "o": o}, gate_act="sigmoid", alpha=0.5, xn=xn, h=h)
        dx, do = at(v["x"], j), at(v["o"], k)
        got = B.block_norm_grad(xn, o, dxn=at(gx, k), dh=at(gh, j), gate_act="sigmoid", alpha=0.5,
                                dx=dx, do=do, **rest)
        ref, size = D.grads(_f64(r["xn"]), _f64(o), _f64(gx), _f64(gh), _f64(v["pre"]),
                            _f64(v["post"]), _f64(v["gate"]), _f64(v["mask"]), gate_act="sigmoid",
                            alpha=0.5)
        for n in ref:
            _within(got[n], ref[n], 2.0 ** -16 * size[n], n)
        for t in (xn, h, dx, do):
            left = t._base.isnan()
            assert left.sum() == 40 and not t.isnan().any()


def test_no_rows():
    v = _inputs(0, 64, BF, BF)
    r = B.block_norm(**v, mxfp4=True)
    assert r["h"].shape == (0, 64) and r["mx"].scales.shape == (0, 1, 512)
    g = B.block_norm_grad(r["xn"], v["o"], dxn=v["x"], dh=r["h"], pre=v["pre"], post=v["post"],
                          gate=v["gate"])
    assert not g["dpre"].any() and not g["dpost"].any() and g["dgate"].shape == (0,)


def _check_grad(v, dxn=True, dh=True, post_norm=True, gate_act="none", alpha=1.0, eps=1e-6, pad=0,
                amp=1e-2, **kw):
    S, T, d = v["x"].dtype, *v["x"].shape
    how = dict(post_norm=post_norm, gate_act=gate_act, alpha=alpha, eps=eps)
    r = B.block_norm(**{**v, "pre": v["pre"]}, **how)
    Bt = r["h"].dtype if "h" in r else v["o"].dtype
    gx = _wide(_rand(90, T, d, amp=amp), pad, S) if dxn else None
    gh = _wide(_rand(91, T, d, amp=amp), pad, Bt) if dh else None
    if v["mask"] is not None:
        for t in (gx, gh):
            if t is not None:
                t[~v["mask"]] = float("nan")
    names = ("o", "pre", "post", "gate", "mask")
    got = B.block_norm_grad(r["xn"], dxn=gx, dh=gh, **{n: v[n] for n in names}, **how, **kw)
    ref, size = D.grads(_f64(r["xn"]), _f64(v["o"]), _f64(gx), _f64(gh), _f64(v["pre"]),
                        _f64(v["post"]), _f64(v["gate"]), _f64(v["mask"]), **how)
    assert set(got) == set(ref)
    for n in ref:
        _within(got[n], ref[n], 2.0 ** -16 * size[n], n)
    assert got["dx"].dtype == S and ("do" not in got or got["do"].dtype == v["o"].dtype)
    return got


@pytest.mark.parametrize("d", [1, 2, 7, 8, 9, 32, 100, 256, 257, 1000, 2560, 2816, 4096, 4104, 8192,
                               8200, 11264, 16384])
def test_gradient_widths(d):
    _check_grad(_inputs(5, d, BF, BF), gate_act="sigmoid", alpha=0.5)


@pytest.mark.parametrize("S,Bt", TYPES)
@pytest.mark.parametrize("d", [96, 1001, 4608, 9000])
def test_gradient_types(S, Bt, d):
    _check_grad(_inputs(9, d, S, Bt, pad=8), alpha=0.7, pad=8)


@pytest.mark.parametrize("T", [1, 2, 33, 607, 609, 5000])
def test_gradient_lengths(T):
    _check_grad(_inputs(T, 200, BF, BF, mask=True), gate_act="sigmoid")


@pytest.mark.parametrize("post_norm", [True, False])
@pytest.mark.parametrize("post", [True, False])
@pytest.mark.parametrize("gate", [None, "none", "sigmoid"])
@pytest.mark.parametrize("dxn,dh", [(True, True), (True, False), (False, True)])
def test_gradient_choices(post_norm, post, gate, dxn, dh):
    v = _inputs(40, 264, F16, F16, post=post, gate=gate is not None, mask=True, pad=3)
    _check_grad(v, dxn, dh, post_norm=post_norm, gate_act=gate or "none", alpha=1.5, eps=1e-5, pad=5)


@pytest.mark.parametrize("dxn", [True, False])
def test_gradient_of_a_norm_alone(dxn):
    v = _inputs(70, 1000, BF, BF, o=False, mask=True)
    _check_grad(v, dxn, True, alpha=3.0)  # alpha is not looked at without o


def test_gradient_of_a_block_without_a_norm_behind_it():
    _check_grad(_inputs(70, 1000, BF, BF, pre=False), True, False)


def test_gradient_in_place_without_weights():
    v = _inputs(50, 640, F32, BF)
    r = B.block_norm(**v)
    dxn, dh = _rand(90, 50, 640).cuda(), _rand(91, 50, 640).to("cuda", BF)
    names = ("pre", "post", "gate")
    how = {n: v[n] for n in names}
    want = B.block_norm_grad(r["xn"], v["o"], dxn=dxn, dh=dh, **how)
    got = B.block_norm_grad(r["xn"], v["o"], dxn=dxn, dh=dh, dx=dxn, do=dh, weights=False, **how)
    assert "dpre" not in got and "dpost" not in got
    assert got["dx"] is dxn and torch.equal(dxn, want["dx"])
    assert got["do"] is dh and torch.equal(dh, want["do"])
    assert torch.equal(got["dgate"], want["dgate"])


def test_the_same_bits_every_time():
    v = _inputs(3000, 2560, BF, BF, mask=True)
    r = B.block_norm(**v, mxfp4=True)
    dxn, dh = _rand(90, 3000, 2560).to("cuda", BF), _rand(91, 3000, 2560).to("cuda", BF)
    names = ("o", "pre", "post", "gate", "mask")
    how = {n: v[n] for n in names}
    g = B.block_norm_grad(r["xn"], dxn=dxn, dh=dh, **how)
    for _ in range(3):
        again = B.block_norm(**v, mxfp4=True)
        for n in ("xn", "h"):
            assert torch.equal(again[n], r[n])
        assert torch.equal(again["mx"].codes, r["mx"].codes)
        more = B.block_norm_grad(r["xn"], dxn=dxn, dh=dh, **how)
        assert all(torch.equal(more[n], g[n]) for n in g)


def test_refusals():
    v = _inputs(4, 64, BF, BF)
    for bad in (dict(o=v["o"].half()), dict(pre=v["pre"].half()), dict(post=v["post"][:32]),
                dict(gate=v["gate"][:2]), dict(gate=v["gate"].bfloat16()),
                dict(mask=torch.ones(3, dtype=torch.bool, device="cuda")),
                dict(o=v["o"].t().contiguous().t()), dict(h_dtype=F16), dict(gate_act="tanh"),
                dict(o=None), dict(pre=None, mxfp4=True), dict(pre=v["pre"].cpu())):
        with pytest.raises(ValueError):
            B.block_norm(**{**v, **bad})
    with pytest.raises(ValueError):
        B.block_norm(v["x"].double(), pre=v["pre"])
    with pytest.raises(B.MoeError):
        B.block_norm(torch.zeros(1, 16385, device="cuda"), pre=torch.ones(16385, device="cuda"))
    with pytest.raises(ValueError):  # rows of MXFP4 come in blocks of 32
        B.block_norm(torch.zeros(1, 40, device="cuda"), pre=torch.ones(40, device="cuda"), mxfp4=True)
    g = dict(dxn=v["x"], dh=v["o"], pre=v["pre"], post=v["post"], gate=v["gate"])
    for bad in (dict(dxn=None, dh=None), dict(pre=None), dict(dxn=v["x"].float()),
                dict(dh=v["o"].float()), dict(dh=v["o"][:2]), dict(do=v["o"].float()),
                dict(dx=v["x"][:, :32])):
        with pytest.raises(ValueError):
            B.block_norm_grad(v["x"], v["o"], **{**g, **bad})
    with pytest.raises(B.MoeError):
        B.block_norm_grad(v["x"], v["o"], **g, ws=torch.empty(8, dtype=torch.uint8, device="cuda"))
