"""The block that runs router, experts and dense projections together against
the 64-bit definitions, and a training step of its router."""
import numpy as np
import pytest
import torch

import oracle
from oracle import router as R

from helpers import host16, host_f

from moe_prefill_routing_gb300 import binding as B
from moe_prefill_routing_gb300.block import MoeBlock

pytestmark = pytest.mark.gpu


def _block(T, d, E, k, f, h, seed, **kw):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s, amp=1.0: (amp * torch.randn(*s, generator=g)).to("cuda", torch.bfloat16)  # noqa: E731
    layer = B.MoeLayer(r(E, d, f, amp=0.05), r(E, d, f, amp=0.05), r(E, f, d, amp=0.05))
    up, down = (r(h, d, amp=0.05), r(d, h, amp=0.05)) if h else (None, None)
    return MoeBlock(layer, r(E, d, amp=0.1), k, up=up, down=down, **kw), r(T, d)


@pytest.mark.parametrize("T,d,E,k,f,h", [(1, 128, 16, 2, 64, 0), (7, 128, 16, 2, 64, 192),
                                          (300, 192, 24, 3, 64, 328)])
def test_block_forward(T, d, E, k, f, h):
    block, x = _block(T, d, E, k, f, h, seed=T)
    r = block.route(x)
    # the router in 64 bits; its choice may differ where logits tie in fp32
    logits = host_f(x) @ host_f(block.Wr).T
    ref = R.route(logits, k)
    top = -np.sort(-logits, axis=1)[:, :k + 1]
    clear = (top[:, :-1] - top[:, 1:] > 1e-5).all(1)
    assert clear.mean() > 0.9
    assert np.array_equal(r["ids"].cpu().numpy()[clear], ref["ids"][clear])
    # the rest from the chosen ids: the layer's tolerance, 1e-2 of the largest value
    y = oracle.layer(host16(x), r["ids"].cpu().numpy(), r["w"].cpu().numpy(),
                     host16(block.layer.Wg), host16(block.layer.Wu), host16(block.layer.Wd))
    y = y + host_f(x)
    if h:
        hid, _ = R.linear(host_f(x), host_f(block.up), act_name="gelu_tanh")
        y, _ = R.linear(hid, host_f(block.down), residual=y)
    got = host_f(block.forward(x))
    # three roundings to bf16 on the way (experts' sum, residual, hidden) of 2^-8 each
    assert np.max(np.abs(got - y)) <= 2.5e-2 * np.max(np.abs(y)) + 1e-3


def test_block_masked_tokens_get_their_residual_alone():
    block, x = _block(40, 128, 16, 2, 64, 0, seed=3)
    mask = torch.ones(40, dtype=torch.bool, device="cuda")
    mask[5:9] = False
    out = block.forward(x, mask)
    assert torch.equal(out[5:9], x[5:9]) and not torch.equal(out[0], x[0])


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_router_step_lowers_its_losses(score):
    block, x = _block(400, 128, 32, 4, 64, 0, seed=5, score=score)
    x = x + 0.5  # a common part, so that some experts are preferred
    first, _ = block.train_router(x, lr=0.0, balance=1.0, z=0.01)
    for _ in range(30):
        last, dx = block.train_router(x, lr=0.5, balance=1.0, z=0.01)
    assert float(last[0] + 0.01 * last[1]) < float(first[0] + 0.01 * first[1])
    assert tuple(dx.shape) == (400, 128) and bool(dx.isfinite().all())


def test_router_gradient_against_differences():
    # d(balance + z) / dWr along a direction, by central differences of the
    # block's own losses in fp32 with the counts as they are: steps of 2^-4 in
    # bf16-exact weights, fp32 losses good to 1e-5 of themselves
    block, x = _block(200, 64, 12, 3, 64, 0, seed=7)
    q = lambda t: (torch.round(t.float() * 64) / 64).to(torch.bfloat16)  # noqa: E731
    x, block.Wr = q(x).clamp(-2, 2), q(block.Wr)
    g = torch.Generator().manual_seed(1)
    v = torch.sign(torch.randn(12, 64, generator=g)).cuda()
    r = block.route(x, stats=True)
    dloss = torch.tensor([0.0, 1.0], device="cuda")  # z alone: no counts in it
    dl = B.route_grad(r["logits"], r["ids"], r["counts"], dloss=dloss, **block.how)
    _, dW, _ = B.linear_grad(x, block.Wr, dl, need=(False, True, False), dw_dtype=torch.float32)
    h = 2.0 ** -6
    z = []
    W0 = block.Wr.clone()
    for s in (h, -h):
        block.Wr = (W0.float() + s * v).to(torch.bfloat16)
        z.append(float(block.route(x, stats=True)["loss"][1]))
    want = (z[0] - z[1]) / (2 * h)
    got = float((dW.double() * v.double()).sum())
    mag = float(dW.double().abs().sum())
    # dlogits is rounded to bf16 for the product (2^-8); h^2 of a third
    # derivative; the losses' rounding over h
    assert abs(got - want) <= (2.0 ** -8 + h) * mag + 1e-5 * z[0] / h
