"""Blocks with norms, gates and a dense expert in MXFP4, one after another: the
pass between two blocks gives the same bits as its parts, the whole is the
definition's, the router's training step goes through the norm."""
import numpy as np
import pytest
import torch

import oracle
from oracle import block as D
from oracle import router as R

from helpers import host16, host_f

from moe_prefill_routing_gb300 import binding as B
from moe_prefill_routing_gb300.block import MoeBlock, run_blocks

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


def _blocks(count, d, E, k, f, h, seed, mx=True, gate=True, post=True, alpha=0.8):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s, amp=1.0: (amp * torch.randn(*s, generator=g)).to("cuda", BF)  # noqa: E731
    made = []
    for _ in range(count):
        layer = B.MoeLayer(r(E, d, f, amp=0.05), r(E, d, f, amp=0.05), r(E, f, d, amp=0.05))
        up, down = (r(h, d, amp=0.05), r(d, h, amp=0.05)) if h else (None, None)
        if h and mx:
            up, down = B.quantize_rows_mxfp4(up), B.quantize_rows_mxfp4(down)
        made.append(MoeBlock(layer, r(E, d, amp=0.1), k, up=up, down=down,
                             pre=1 + r(d, amp=0.1).float(), alpha=alpha,
                             post=1 + r(d, amp=0.1).float() if post else None,
                             gate=r(1, d, amp=0.1) if gate else None))
    return made


def _x(T, d, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(T, d, generator=g).to("cuda", dtype)


def _step_by_step(blocks, x, mask):
    for b in blocks:
        n = B.block_norm(x, pre=b.pre, mask=mask, h_dtype=BF)
        h = n["h"]
        r = b.route(h, mask)
        y = b.layer.forward(h, r["ids"], r["w"])
        if isinstance(b.up, B.Mxfp4Rows):
            hid = B.linear_mxfp4(B.quantize_rows_mxfp4(h), b.up, act="gelu_tanh")
            y = B.linear_mxfp4(B.quantize_rows_mxfp4(hid), b.down, residual=y, out_dtype=BF)
        elif b.up is not None:
            y = B.linear(B.linear(h, b.up, act="gelu_tanh"), b.down, residual=y)
        g = None if b.gate is None else B.linear(h, b.gate, out_dtype=F32).view(-1)
        x = B.block_norm(x, y, post=b.post, gate=g, mask=mask, post_norm=b.post is not None,
                         gate_act="sigmoid", alpha=b.alpha)["xn"]
    return x


@pytest.mark.parametrize("T", [1, 3, 40, 200])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("kw", [dict(), dict(mx=False), dict(gate=False, post=False, alpha=1.0),
                                dict(h=0)])
def test_several_blocks_are_their_parts(T, dtype, kw):
    blocks = _blocks(3, 128, 16, 2, 64, kw.get("h", 192), seed=T,
                     **{n: v for n, v in kw.items() if n != "h"})
    x = _x(T, 128, dtype, T)
    keep = x.clone()
    for mask in (None, (torch.arange(T) % 3 != 1).cuda()):
        got = run_blocks(blocks, x, mask)
        assert got.dtype == dtype and torch.equal(x, keep)
        assert torch.equal(got, _step_by_step(blocks, x, mask))
        if mask is not None:
            assert not got[~mask].any()
    assert torch.equal(blocks[0].forward(x), _step_by_step(blocks[:1], x, None))
    assert blocks[0].status() == 0 and torch.equal(run_blocks([], x), x)


@pytest.mark.parametrize("T,d,E,k,f,h", [(5, 128, 16, 2, 64, 192), (260, 192, 24, 3, 64, 320)])
def test_a_block_is_the_definition(T, d, E, k, f, h):
    b, = _blocks(1, d, E, k, f, h, seed=T)
    x = _x(T, d, F32, T)
    # what the block decides by rounding is taken as it came out: h, the choice
    # of experts and the dense expert's hidden rows in MXFP4
    n = B.block_norm(x, pre=b.pre, h_dtype=BF, mxfp4=True)
    want_h = D.normed(host_f(x), host_f(b.pre))
    assert np.max(np.abs(host_f(n["h"]) - want_h)) <= 2.0 ** -7.9 * np.max(np.abs(want_h))
    r = b.route(n["h"])
    y = oracle.layer(host16(n["h"]), r["ids"].cpu().numpy(), r["w"].cpu().numpy(),
                     host16(b.layer.Wg), host16(b.layer.Wu), host16(b.layer.Wd))
    value = lambda q: D.mx_values(*D.mx_unpack(q.codes.cpu().numpy(), q.scales.cpu().numpy()))  # noqa: E731
    hid, _ = R.linear(value(n["mx"]), value(b.up), act_name="gelu_tanh")
    own = B.linear_mxfp4(n["mx"], b.up, act="gelu_tanh")
    assert np.max(np.abs(host_f(own) - hid)) <= 2.0 ** -7.9 * np.max(np.abs(hid))
    y, _ = R.linear(value(B.quantize_rows_mxfp4(own)), value(b.down), residual=y)
    gate = host_f(n["h"]) @ host_f(b.gate)[0]
    out = D.stream(host_f(x), y, host_f(b.post), gate, gate_act="sigmoid", alpha=b.alpha)
    got = host_f(b.forward(x))
    # the experts' sum to 1e-2 of its largest value, and its own rounding to bf16;
    # the norm divides both by the same
    assert np.max(np.abs(got - out)) <= 2.5e-2 * np.max(np.abs(out - b.alpha * host_f(x))) + 1e-3


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("masked", [False, True])
def test_the_routers_step_goes_through_the_norm(dtype, masked):
    b, = _blocks(1, 192, 24, 3, 64, 0, seed=8)
    plain = MoeBlock(b.layer, b.Wr.clone(), b.k)
    x = _x(150, 192, dtype, 9)
    mask = (torch.arange(150) % 4 != 2).cuda() if masked else None
    h = B.block_norm(x, pre=b.pre, mask=mask, h_dtype=BF)["h"]
    scale = 2.0 ** 14
    if masked:
        x[~mask] = float("nan")
    loss, dx = b.train_router(x, lr=0.1, mask=mask, grad_scale=scale)
    want, dh = plain.train_router(h, lr=0.1, mask=mask, grad_scale=scale)
    assert torch.equal(loss, want) and torch.equal(b.Wr, plain.Wr)
    xd = host_f(x) if mask is None else np.where(mask.cpu().numpy()[:, None], host_f(x), 0.0)
    ref, size = D.grads(xd, dh=host_f(dh), pre=host_f(b.pre),
                        mask=None if mask is None else mask.cpu().numpy())
    half = torch.finfo(dtype).eps / 2
    tol = 2.0 ** -16 * size["dx"]
    assert dx.dtype == dtype
    assert np.all(np.abs(host_f(dx) - ref["dx"]) <= tol + half * (np.abs(ref["dx"]) + tol))
    if masked:
        assert not dx[~mask].any()


def test_refusals():
    b, = _blocks(1, 128, 16, 2, 64, 192, seed=1)
    with pytest.raises(ValueError):
        MoeBlock(b.layer, b.Wr, 2, post=b.post)
    with pytest.raises(ValueError):
        MoeBlock(b.layer, b.Wr, 2, alpha=0.5)
    with pytest.raises(ValueError):
        MoeBlock(b.layer, b.Wr, 2, up=b.up, down=torch.empty(128, 192, dtype=BF, device="cuda"))
    with pytest.raises(ValueError):
        run_blocks([MoeBlock(b.layer, b.Wr, 2)], _x(4, 128, BF, 1))
    with pytest.raises(ValueError):
        run_blocks([b], _x(4, 128, torch.float16, 1))
    other, = _blocks(1, 128, 16, 2, 64, 0, seed=1)
    other.eps = 1e-5
    with pytest.raises(ValueError):
        run_blocks([b, other], _x(4, 128, BF, 1))


def test_a_plain_block_with_a_dense_expert_in_mxfp4():
    b, = _blocks(1, 128, 16, 2, 64, 192, seed=4)
    plain = MoeBlock(b.layer, b.Wr, 2, up=b.up, down=b.down)
    x = _x(60, 128, BF, 5)
    r = plain.route(x)
    y = plain.layer.forward(x, r["ids"], r["w"]).add_(x)
    hid = B.linear_mxfp4(x, b.up, act="gelu_tanh")
    assert torch.equal(plain.forward(x), B.linear_mxfp4(hid, b.down, residual=y, out_dtype=BF))
