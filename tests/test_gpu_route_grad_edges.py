"""moe_route_grad where slots have no weight, experts are closed, and the
gradients handed to it are no numbers there."""
import pytest
import torch

from moe_prefill_routing_gb300 import binding as B

pytestmark = pytest.mark.gpu


def _case(E, k, dtype=torch.float32, T=37):
    g = torch.Generator().manual_seed(E + k)
    l = 2 * torch.randn(T, E, generator=g)
    l[torch.rand(T, E, generator=g) < 0.2] = -float("inf")
    l[3, k // 2:] = -float("inf")  # fewer open experts than slots
    l[4] = -float("inf")
    return l.to(dtype).cuda()


@pytest.mark.parametrize("E,k", [(8, 4), (64, 6), (200, 40), (512, 10), (700, 5), (3000, 40)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("norm", [True, False])
def test_dw_of_slots_without_weight_is_not_looked_at(E, k, score, norm):
    l = _case(E, k)
    kw = dict(score=score, norm=norm)
    r = B.route(l, k, **kw)
    ids = r["ids"].clone()
    ids[0, 1] = -1            # a slot that the caller dropped
    ids[1, 0] = E + 7         # outside
    ids[2, 2] = -5
    closed = (l[6] == -float("inf")).nonzero()[0]
    ids[6, 3] = closed.to(torch.int32)  # a closed expert
    ok = (ids >= 0) & (ids < E)
    ok &= l.gather(1, ids.clamp(0, E - 1).long()) > -float("inf")
    assert int((~ok).sum()) > 4
    dw = torch.randn(ids.shape, generator=torch.Generator().manual_seed(1)).cuda()
    dloss = torch.tensor([0.7, -0.4], device="cuda")
    want = B.route_grad(l, ids, r["counts"], dw=torch.where(ok, dw, 0.0), dloss=dloss, **kw)
    assert bool(want.isfinite().all())
    for poison in (float("nan"), float("inf"), -float("inf")):
        got = B.route_grad(l, ids, r["counts"], dw=torch.where(ok, dw, poison), dloss=dloss, **kw)
        assert torch.equal(got, want), poison


@pytest.mark.parametrize("E,k,dtype", [(64, 6, torch.float32), (512, 10, torch.bfloat16),
                                       (1500, 12, torch.float32)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("norm", [True, False])
def test_closed_experts_gradient_is_zero_whatever_comes_in(E, k, dtype, score, norm):
    # an overflowed loss scale: infinities and NaN in dloss or in dw of a used slot
    l = _case(E, k, dtype)
    kw = dict(score=score, norm=norm)
    r = B.route(l, k, **kw)
    inf, nan = float("inf"), float("nan")
    closed = l == -inf
    dw = torch.ones(r["ids"].shape, device="cuda")
    for a, b, c in ((inf, 1.0, 1.0), (1.0, -inf, 1.0), (nan, 1.0, 1.0), (1.0, 1.0, inf),
                    (1.0, 1.0, nan), (3e38, 3e38, -3e38)):
        dw[:, 0] = c
        g = B.route_grad(l, r["ids"], r["counts"], dw=dw, dloss=torch.tensor([a, b], device="cuda"),
                         **kw)
        assert bool((g[closed] == 0).all()), (a, b, c)
        assert not bool(g.isfinite().all()) or a == 3e38


@pytest.mark.parametrize("E,k", [(14, 1), (200, 1), (512, 1), (900, 1), (40, 3), (2500, 5)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_a_weight_that_is_alone_has_no_gradient(E, k, score):
    # renormalised over itself it is `scale` whatever the logits: dw adds
    # nothing, beside losses a million times smaller
    l = torch.randn(300, E, generator=torch.Generator().manual_seed(E))
    if k > 1:  # one open expert a token
        keep = torch.randint(E, (300, 1), generator=torch.Generator().manual_seed(1))
        l = torch.full_like(l, -float("inf")).scatter(1, keep, l.gather(1, keep))
    l = l.cuda()
    r = B.route(l, k, score=score, scale=2.5)
    dw = torch.randn(300, k, generator=torch.Generator().manual_seed(2)).cuda()
    dloss = torch.tensor([1e-4, 1e-6], device="cuda")
    kw = dict(dloss=dloss, score=score, scale=2.5)
    got = B.route_grad(l, r["ids"], r["counts"], dw=dw, **kw)
    assert torch.equal(got, B.route_grad(l, r["ids"], r["counts"], **kw))
    assert bool((B.route_grad(l, r["ids"], dw=dw, score=score, scale=2.5) == 0).all())
