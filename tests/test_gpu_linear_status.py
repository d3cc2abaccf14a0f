"""What moe_linear and moe_route report without a status word of the caller's,
and the stop of a linear kernel whose wait runs out: no GPU fault, a CTA's
first stage expects 16 bytes that never arrive, so its bounded waits run out
(about 2 s) and it stops; the context keeps working."""
import time

import pytest
import torch

from moe_prefill_routing_gb300 import binding as B

pytestmark = pytest.mark.gpu


def _rand(seed, *shape, amp=1.0):
    g = torch.Generator().manual_seed(seed)
    return (amp * torch.randn(*shape, generator=g)).to("cuda", torch.bfloat16)


# few tokens, one CTA a tile; few tokens, split over a cluster; pairs of CTAs;
# pairs, split over a cluster.  `lost`: rows and columns of the stopped tile
@pytest.mark.parametrize("T,K,N,cta,lost", [
    (16, 192, 512, 1, (slice(0, 16), slice(128, 256))),
    (16, 4096, 512, 8, None),
    (3000, 200, 4000, 4, None),
    (300, 2560, 512, 2, None)])
@pytest.mark.parametrize("own", [True, False])
def test_a_wait_that_runs_out_is_reported(T, K, N, cta, lost, own):
    x, W = _rand(1, T, K), _rand(2, N, K, amp=K ** -0.5)
    want = B.linear(x, W)
    torch.cuda.synchronize()
    assert B.take_status() == 0
    word = torch.zeros(1, dtype=torch.int32, device="cuda") if own else None
    t0 = time.time()
    y = B.selftest_linear_wait_limit(x, W, cta, word)
    torch.cuda.synchronize()
    assert 1.0 < time.time() - t0 < 60.0
    taken = B.take_status()
    if own:
        assert int(word.item()) == B.STATUS_TIMEOUT and taken == 0
    else:
        assert taken == B.STATUS_TIMEOUT and B.take_status() == 0  # cleared
    if lost:  # the other tiles are what they should be
        keep = torch.ones((T, N), dtype=torch.bool, device="cuda")
        keep[lost] = False
        assert torch.equal(y[keep], want[keep])
    assert torch.equal(B.linear(x, W), want) and B.take_status() == 0


def test_calls_with_a_status_word_leave_it_alone():
    x, W, dy = _rand(1, 200, 128), _rand(2, 96, 128), _rand(3, 200, 96)
    word = torch.zeros(1, dtype=torch.int32, device="cuda")
    y = B.linear(x, W, status=word)
    g = B.linear_grad(x, W, dy, status=word)
    assert torch.equal(y, B.linear(x, W))
    assert all(torch.equal(a, b) for a, b in zip(g, B.linear_grad(x, W, dy)))
    assert int(word.item()) == 0


@pytest.mark.parametrize("T", [3, 500])
def test_route_without_a_workspace_reports_bad_logits(T):
    l = torch.randn(T, 96, generator=torch.Generator().manual_seed(1)).cuda()
    B.take_status()
    B.route(l, 4, stats=False)
    assert B.take_status() == 0
    l[T - 1, 7] = float("nan")
    B.route(l, 4, stats=False)
    B.route(l[:1], 4, stats=False)
    assert B.take_status() == B.STATUS_BAD_LOGIT and B.take_status() == 0
    ws = B.route(l, 4)["ws"]
    assert B.read_status(ws) == B.STATUS_BAD_LOGIT and B.take_status() == 0
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        B.route(l, 4, stats=False)
        assert B.take_status() == B.STATUS_BAD_LOGIT


def test_words_and_workspaces_are_checked():
    x, W = _rand(1, 20, 64), _rand(2, 24, 64)
    dy, l = _rand(3, 20, 24), torch.zeros(20, 32, device="cuda")
    cpu = torch.zeros(1, dtype=torch.int32)
    for bad in (cpu, cpu.cuda().to(torch.int8), cpu.cuda()[:0]):
        with pytest.raises(ValueError, match="status"):
            B.linear(x, W, status=bad)
        with pytest.raises(ValueError, match="status"):
            B.linear_grad(x, W, dy, status=bad)
    with pytest.raises(ValueError, match="ws"):
        B.linear_grad(x, W, dy, ws=torch.empty(1 << 20, dtype=torch.uint8))
    with pytest.raises(ValueError, match="ws"):
        B.route(l, 2, ws=torch.empty(1 << 20, dtype=torch.uint8))
    # a workspace of another element type counts in bytes
    n = B.linear_grad_workspace_bytes(20, 24, torch.bfloat16, torch.bfloat16)
    B.linear_grad(x, W, dy, ws=torch.empty((n + 3) // 4, dtype=torch.int32, device="cuda"))
    n = B.route_workspace_bytes(20, 32)
    B.route(l, 2, ws=torch.empty((n + 3) // 4, dtype=torch.int32, device="cuda"))
