"""moe_route and moe_route_grad against the 64-bit definitions.

Ids and counts have to be equal.  With a bias the keys are computed scores,
so tokens whose first k + 1 keys lie within 1e-5 of one another are left out
of the inputs (their logits are redrawn).  Exponentials of fp32 arguments up
to 30 in magnitude are good to 40 units of 2^-24 (2.4e-6), a ratio of sums of
them to twice that: weights and probabilities are held to 1e-5 of
themselves, losses and gradients to 1e-5 of the magnitudes they are sums of."""
import numpy as np
import pytest
import torch

from oracle import router as R

from moe_prefill_routing_gb300 import binding as B

pytestmark = pytest.mark.gpu

REL = 1e-5


def _logits(T, E, seed, dtype=torch.float32, closed=0.0, spread=2.0):
    g = torch.Generator().manual_seed(seed)
    l = spread * torch.randn(T, E, generator=g) + torch.randn(E, generator=g)
    l = l.to(dtype)
    if closed:
        l[torch.rand(T, E, generator=g) < closed] = -float("inf")
    return l


def _apart(l, k, bias, score, mask):
    """Redraws tokens whose choice depends on the rounding of a score."""
    for seed in range(50):
        keys = R.route(l.double().numpy(), k, bias=bias, mask=mask, score=score)["keys"]
        top = -np.sort(-keys, axis=1)[:, :k + 1]
        with np.errstate(invalid="ignore"):
            near = np.flatnonzero((top[:, :-1] - top[:, 1:] < 1e-5).any(1))
        if near.size == 0:
            return l
        l[near] = _logits(near.size, l.shape[1], 1000 + seed, l.dtype)
    raise AssertionError("no inputs with keys apart")


def _np(t):
    return t.detach().double().cpu().numpy()


def _check(T, E, k, seed=0, dtype=torch.float32, score="softmax", norm=True, scale=1.0,
           bias=False, masked=0.0, closed=0.0, spread=2.0, pad=0):
    l = _logits(T, E, seed, dtype, closed, spread)
    rng = np.random.default_rng(seed)
    mask = (rng.random(T) >= masked).astype(np.uint8) if masked else None
    b = (0.5 * rng.standard_normal(E)).astype(np.float32) if bias else None
    if bias:
        l = _apart(l, k, b.astype(np.float64), score, mask)
    if mask is not None:
        l[torch.from_numpy(mask == 0)] = float("nan")
    kw = dict(score=score, norm=norm, scale=scale)
    ref = R.route(l.double().numpy(), k, bias=None if b is None else b.astype(np.float64),
                  mask=mask, **kw)
    wide = torch.full((T, E + pad), float("nan"), dtype=dtype, device="cuda")
    wide[:, :E] = l.cuda()
    dl = wide[:, :E]
    dm = None if mask is None else torch.from_numpy(mask).cuda()
    db = None if b is None else torch.from_numpy(b).cuda()
    r = B.route(dl, k, bias=db, mask=dm, **kw)
    assert B.read_status(r["ws"]) == 0
    assert np.array_equal(r["ids"].cpu().numpy(), ref["ids"])
    assert np.array_equal(r["counts"].cpu().numpy(), ref["counts"])
    assert np.all(np.abs(_np(r["w"]) - ref["w"]) <= REL * ref["w"] + 1e-37)
    assert np.all(np.abs(_np(r["prob"]) - ref["prob"]) <= REL * ref["prob"] + 1e-37)
    assert np.all(np.abs(_np(r["loss"]) - ref["loss"]) <= REL * np.abs(ref["loss"]))
    bare = B.route(dl, k, bias=db, mask=dm, stats=False, **kw)
    assert torch.equal(bare["ids"], r["ids"]) and torch.equal(bare["w"], r["w"])

    dw = rng.standard_normal((T, k)).astype(np.float32)
    dloss = np.array([0.7, -0.4], dtype=np.float32)
    g = B.route_grad(dl, r["ids"], r["counts"], dw=torch.from_numpy(dw).cuda(),
                     dloss=torch.from_numpy(dloss).cuda(), mask=dm, **kw)
    assert g.dtype == dtype
    args = (l.double().numpy(), ref["ids"], ref["counts"])
    rg = R.route_grad(*args, dw.astype(np.float64), dloss.astype(np.float64), mask=mask, **kw)
    # magnitudes of the parts: weights' (scale |dw| over the row), balance, z
    n = max(1, int(ref["counts"][E]))
    mag = (scale * np.abs(dw).sum(1, keepdims=True) + 2 * 0.4 * np.sqrt(ref["loss"][1] + 100) / n
           + 0.7 * E * ref["counts"][:E].max() / (n * k) / n)
    half = torch.finfo(dtype).eps / 2
    small = 2.0 ** -25 if dtype == torch.float16 else 1e-37
    assert np.all(np.abs(_np(g) - rg) <= REL * mag + half * np.abs(rg) + small)


@pytest.mark.parametrize("T,E,k", [
    (1, 1, 1), (1, 512, 10), (3, 2, 2), (5, 31, 4), (8, 32, 1), (9, 33, 33), (64, 64, 6),
    (100, 65, 8), (33, 128, 8), (40, 129, 16), (257, 256, 8), (50, 300, 64), (130, 512, 10),
    (40, 512, 256), (40, 500, 40), (20, 513, 10), (12, 1000, 33), (9, 1025, 8), (6, 4096, 256)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_route_shapes(T, E, k, score):
    _check(T, E, k, score=score)
    _check(T, E, k, score=score, norm=False, scale=2.5, closed=0.3, masked=0.3, seed=1, pad=3)


@pytest.mark.parametrize("T,E,k", [(600, 1024, 8), (70, 1500, 200), (300, 2048, 140), (37, 2049, 3)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_route_many_experts(T, E, k, score):
    _check(T, E, k, score=score, masked=0.2, seed=4)
    _check(T, E, k, score=score, norm=False, closed=0.3, dtype=torch.bfloat16, seed=5, pad=8)
    _check(T, E, k, score=score, bias=True, scale=2.5, seed=6)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("norm", [True, False])
def test_route_selection_bias(score, norm):
    _check(300, 64, 6, score=score, norm=norm, bias=True, scale=2.5)
    _check(200, 200, 8, score=score, norm=norm, bias=True, closed=0.2, masked=0.1, seed=2)
    _check(20, 700, 8, score=score, norm=norm, bias=True, seed=3)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_route_16_bit_logits_with_ties(dtype, score):
    _check(500, 128, 8, dtype=dtype, score=score, masked=0.1)
    _check(100, 600, 8, dtype=dtype, score=score, closed=0.5)


def test_route_far_apart_logits():
    # chosen experts far below the maximum (a bias forces them) keep their ratios
    E, k = 40, 4
    l = torch.full((3, E), -60.0)
    l[:, 0] = 30.0
    l[:, 5], l[:, 6] = -90.0, -91.0
    b = torch.zeros(E)
    b[5], b[6], b[7], b[8] = 9.0, 8.0, 7.0, 6.0
    for score in ("softmax", "sigmoid"):
        r = B.route(l.cuda(), k, bias=b.cuda(), score=score)
        ref = R.route(l.double().numpy(), k, bias=b.double().numpy(), score=score)
        assert r["ids"].cpu().numpy().tolist() == ref["ids"].tolist() == [[5, 6, 7, 8]] * 3
        assert np.all(np.abs(_np(r["w"]) - ref["w"]) <= 2e-5 * ref["w"])


def test_route_all_equal_and_signed_zeros():
    l = torch.zeros(4, 70)
    l[1, ::2] = -0.0
    l[2] = -1e30
    l[3] = 3e38
    r = B.route(l.cuda(), 5)
    assert r["ids"].cpu().tolist() == [[0, 1, 2, 3, 4]] * 4
    assert torch.allclose(r["w"].cpu(), torch.full((4, 5), 0.2), rtol=REL, atol=0)


def test_route_nobody_takes_part():
    l = torch.full((6, 48), float("nan"), device="cuda")
    r = B.route(l, 3, mask=torch.zeros(6, dtype=torch.bool, device="cuda"))
    assert B.read_status(r["ws"]) == 0
    assert bool((r["ids"] == -1).all()) and bool((r["w"] == 0).all())
    assert bool((r["counts"] == 0).all()) and bool((r["prob"] == 0).all())
    assert bool((r["loss"] == 0).all())
    g = B.route_grad(l, r["ids"], r["counts"], dw=torch.ones(6, 3, device="cuda"),
                     dloss=torch.ones(2, device="cuda"),
                     mask=torch.zeros(6, dtype=torch.bool, device="cuda"))
    assert bool((g == 0).all())
    closed = torch.full((6, 48), -float("inf"), device="cuda")
    assert int(B.route(closed, 3)["counts"].sum()) == 0


def test_route_reports_logits_that_are_no_numbers():
    l = _logits(50, 96, 4)
    l[7, 11] = float("nan")
    l[9, 3] = float("inf")
    ref = R.route(l.double().numpy(), 5)
    r = B.route(l.cuda(), 5)
    assert B.read_status(r["ws"]) == B.STATUS_BAD_LOGIT
    lean = B.route(l.cuda(), 5, stats=False, ws=torch.empty_like(r["ws"]))
    assert B.read_status(lean["ws"]) == B.STATUS_BAD_LOGIT and "ws" not in B.route(
        l.cuda(), 5, stats=False)
    assert np.array_equal(r["ids"].cpu().numpy(), ref["ids"])
    ok = B.route(_logits(50, 96, 4).cuda(), 5, ws=r["ws"])
    assert B.read_status(ok["ws"]) == 0


def test_route_no_tokens():
    r = B.route(torch.empty((0, 20), device="cuda"), 4)
    assert tuple(r["ids"].shape) == (0, 4) and bool((r["counts"] == 0).all())
    assert bool((r["loss"] == 0).all()) and B.read_status(r["ws"]) == 0
    assert tuple(B.route_grad(torch.empty((0, 20), device="cuda"), r["ids"]).shape) == (0, 20)


def test_route_many_tokens_same_bits_every_time():
    l = _logits(40000, 96, 5).cuda()
    a, b = B.route(l, 6), B.route(l, 6)
    for n in ("ids", "w", "counts", "prob", "loss"):
        assert torch.equal(a[n], b[n]), n
    assert int(a["counts"][:96].sum()) == 240000 and int(a["counts"][96]) == 40000
    # the definition on the whole, in 64 bits on the GPU
    p = torch.softmax(l.double(), 1).mean(0)
    assert torch.allclose(a["prob"].double(), p, rtol=REL, atol=0)
    want = 96 * float((a["counts"][:96].double() / 240000 * p).sum())
    assert abs(float(a["loss"][0]) - want) <= REL * want
    z = float(torch.logsumexp(l.double(), 1).square().mean())
    assert abs(float(a["loss"][1]) - z) <= REL * z


def test_route_logits_beyond_31_bit_offsets():
    T, E, ld = 70000, 8, 32768
    big = torch.zeros((T, ld), dtype=torch.bfloat16, device="cuda")
    l = big[:, :E]
    l.copy_(_logits(T, E, 6, torch.bfloat16))
    r = B.route(l, 2)
    ref = R.route(l[-3:].double().cpu().numpy(), 2)
    assert np.array_equal(r["ids"][-3:].cpu().numpy(), ref["ids"])
    g = B.route_grad(l, r["ids"], dw=torch.ones(T, 2, device="cuda"), norm=False, dlogits=l)
    assert g.data_ptr() == l.data_ptr() and bool(g[-3:].isfinite().all())


def test_route_feeds_the_plan():
    l = _logits(64, 16, 8).cuda()
    r = B.route(l, 2)
    p = B.plan(r["ids"], r["w"], 16, 16)
    assert torch.equal(p["counts"], r["counts"][:16]) and B.read_status(p["ws"]) == 0


def test_route_grad_parts_add_up():
    T, E, k = 60, 50, 4
    l = _logits(T, E, 9).cuda()
    r = B.route(l, k)
    dw = torch.randn(T, k, generator=torch.Generator().manual_seed(1)).cuda()
    g0 = torch.tensor([2.0, 0.5], device="cuda")
    both = B.route_grad(l, r["ids"], r["counts"], dw=dw, dloss=g0)
    a = B.route_grad(l, r["ids"], dw=dw)
    b = B.route_grad(l, r["ids"], r["counts"], dloss=g0)
    mag = float(dw.abs().sum(1).max())
    assert float((both - a - b).abs().max()) <= 4 * 2.0 ** -24 * mag
    assert bool((B.route_grad(l, r["ids"]) == 0).all())


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("norm", [True, False])
def test_route_grad_against_differences_of_route(score, norm):
    # along a direction v with |v| <= 1, step h = 2^-6: the central difference
    # is off by h^2/6 of a third derivative (at most a few times the
    # magnitudes summed) and by the weights' 1e-5 over h
    T, E, k, h = 40, 24, 5, 2.0 ** -6
    l = torch.zeros(T, E)
    g = torch.Generator().manual_seed(3)
    for t in range(T):  # logits at least 1/8 apart: the choice stays the same
        l[t] = (torch.randperm(E, generator=g) - E / 2) / 8.0
    v = (2 * torch.rand(T, E, generator=g) - 1)
    dw = torch.randn(T, k, generator=g)
    l, v, dw = l.cuda(), v.cuda(), dw.cuda()
    kw = dict(score=score, norm=norm)
    r, up, down = (B.route(x, k, **kw) for x in (l, l + h * v, l - h * v))
    assert torch.equal(up["ids"], r["ids"]) and torch.equal(down["ids"], r["ids"])
    dloss = torch.tensor([3.0, 0.2], device="cuda")
    value = lambda q: ((q["w"].double() * dw.double()).sum()  # noqa: E731
                       + (q["loss"].double() * dloss.double()).sum())
    want = float((value(up) - value(down)) / (2 * h))
    got = float((B.route_grad(l, r["ids"], r["counts"], dw=dw, dloss=dloss, **kw).double()
                 * v.double()).sum())
    mag = float(dw.abs().sum()) + 3.0 + 0.2 * float(r["loss"][1])
    assert abs(got - want) <= (h * h + 1e-5 / h) * mag
