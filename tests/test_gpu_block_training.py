"""A training step of the block's router against the 64-bit gradient of its own
logits, for both operand types and with the usual loss coefficients; what it
does with padding rows, small steps and weights set in between; its status.

Bounds.  dlogits are held to 1e-5 of the magnitudes they are sums of; an fp32
dWr takes them in two 16-bit pieces (2^-16 of each at most) and sums in fp32
(2^-20 of the magnitudes' sum)."""
import numpy as np
import pytest
import torch

from oracle import router as R

from moe_prefill_routing_gb300 import binding as B
from moe_prefill_routing_gb300.block import MoeBlock

pytestmark = pytest.mark.gpu

BF, F16 = torch.bfloat16, torch.float16


def _rand(seed, *shape, amp=1.0):
    g = torch.Generator().manual_seed(seed)
    return amp * torch.randn(*shape, generator=g)


def _router(T, d, E, k, dtype, **kw):
    x = (_rand(T, T, d) + 0.3).to("cuda", dtype)
    return MoeBlock(None, _rand(E, E, d, amp=0.05).to("cuda", dtype), k, **kw), x


def _np(t):
    return t.detach().double().cpu().numpy()


@pytest.mark.parametrize("T,d,E,k,dtype,kw", [
    (300, 128, 32, 4, BF, {}), (300, 128, 32, 4, F16, dict(score="sigmoid", norm=False, scale=2.5)),
    (1000, 264, 65, 6, F16, {}), (700, 72, 130, 8, BF, dict(score="sigmoid")),
    (2048, 2560, 512, 10, BF, {}), (2048, 2560, 512, 10, F16, {})])
def test_step_is_the_gradient(T, d, E, k, dtype, kw):
    block, x = _router(T, d, E, k, dtype, **kw)
    W0 = block.Wr.clone()
    r = block.route(x, stats=True)
    balance, z, lr, scale = 1e-2, 1e-3, 2.0 ** 10, 2.0 ** 12
    dw = _rand(5, T, k, amp=1e-6)
    loss, dx = block.train_router(x, lr=lr, dw=dw.cuda(), grad_scale=scale)
    assert torch.equal(loss, r["loss"])
    counts = r["counts"].cpu().numpy()
    dl = R.route_grad(_np(r["logits"]), r["ids"].cpu().numpy(), counts, _np(dw),
                      np.array([balance, z]), **block.how)
    xd, Wd, n = _np(x), _np(W0), int(counts[E])
    how = {**dict(scale=1.0), **kw}
    mag = (how["scale"] * np.abs(_np(dw)).sum(1, keepdims=True)
           + 2 * z * np.sqrt(float(loss[1]) + 100) / n
           + balance * E * counts[:E].max() / (n * k) / n) * np.ones_like(dl)
    off = 1e-5 * mag
    dW = dl.T @ xd
    got = (Wd - _np(block._master)) / lr
    bound = (off + (2.0 ** -16 + 2.0 ** -20) * (np.abs(dl) + off)).T @ np.abs(xd)
    bound += 2.0 ** -23 * (np.abs(Wd) + lr * np.abs(dW)) / lr  # the step itself, in fp32
    err = np.abs(got - dW)
    assert np.all(err <= bound), float(np.max(err / bound))
    assert np.linalg.norm(err) < 1e-3 * np.linalg.norm(dW)
    # Wr is those weights in 16 bits
    assert torch.equal(block.Wr, block._master.to(dtype)) and not torch.equal(block.Wr, W0)
    # dx: dlogits in one piece, half a unit of dx's type
    half = torch.finfo(dtype).eps / 2
    ref = scale * (dl @ Wd)
    tol = scale * ((off + (half + 2.0 ** -20) * (np.abs(dl) + off)) @ np.abs(Wd))
    small = torch.finfo(dtype).smallest_normal * half
    assert np.all(np.abs(_np(dx) - ref) <= tol + half * (np.abs(ref) + tol) + small)


@pytest.mark.parametrize("dtype", [BF, F16])
def test_padding_rows_may_hold_anything(dtype):
    T, d, E, k = 200, 128, 24, 3
    mask = torch.ones(T, dtype=torch.bool, device="cuda")
    mask[::7] = False
    out = []
    for fill in (0.0, float("nan"), float("inf"), 6e4):
        block, x = _router(T, d, E, k, dtype)
        x[~mask] = fill
        keep = x.clone()
        loss, dx = block.train_router(x, lr=1.0, mask=mask)
        assert torch.equal(x.isnan(), keep.isnan()) and bool((dx[~mask] == 0).all())
        out.append((loss, dx, block.Wr))
    for o in out[1:]:
        assert all(torch.equal(a, b) for a, b in zip(o, out[0]))
    assert bool(out[0][2].isfinite().all())


def test_small_steps_add_up():
    block, x = _router(400, 64, 16, 2, BF)
    W0 = block.Wr.float()
    block.train_router(x, lr=1.0)
    step = (W0 - block._master).abs().max()  # the first step's largest entry
    block, x = _router(400, 64, 16, 2, BF)
    # steps of at most 1/64 of the least weights' spacing seen, a thousand of them
    lr = float(2.0 ** -14 / 64 / step)
    before = block.Wr.clone()
    for _ in range(1000):
        block.train_router(x, lr=lr)
    moved = (block._master - W0).abs().max()
    assert float(moved) > 5 * 2.0 ** -14
    assert torch.equal(block.Wr, block._master.to(BF)) and not torch.equal(block.Wr, before)


def test_weights_set_between_steps_count():
    block, x = _router(100, 64, 16, 2, BF)
    block.train_router(x, lr=0.3)
    block.Wr[3:5] = 0.25                    # in place
    want = block.Wr.clone()
    block.train_router(x, lr=0.0)
    assert torch.equal(block.Wr, want) and bool((block._master[3:5] == 0.25).all())
    block.Wr = _rand(9, 20, 64).to("cuda", BF)  # another tensor
    want = block.Wr.clone()
    block.train_router(x, lr=0.0)
    assert torch.equal(block.Wr, want) and tuple(block._master.shape) == (20, 64)


def test_status_and_types():
    r = lambda *s: _rand(sum(s), *s, amp=0.05).to("cuda", BF)  # noqa: E731
    block = MoeBlock(B.MoeLayer(r(16, 128, 64), r(16, 128, 64), r(16, 64, 128)), r(16, 128), 2,
                     up=r(192, 128), down=r(128, 192))
    x = r(40, 128)
    block.status()
    block.forward(x)
    assert block.status() == 0
    x[5, 7] = float("nan")
    block.forward(x)
    assert block.status() == B.STATUS_BAD_LOGIT and block.status() == 0
    with pytest.raises(ValueError, match="bfloat16"):
        block.forward(x.half())
