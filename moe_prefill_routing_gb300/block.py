"""A whole mixture-of-experts block on the library: norms, router, routed
experts, a dense expert beside them and the residual; and a training step of the
router.

    python -m moe_prefill_routing_gb300.block      # needs a GB300

``MoeBlock.forward`` is what a model runs per layer (a prefill chunk or a few
decoded tokens), ``run_blocks`` several layers, the norms between two of them in
one pass; ``MoeBlock.train_router`` takes one gradient step that balances the
experts, the experts' weights fixed.
"""
from __future__ import annotations

import torch

from . import binding as B


class MoeBlock:
    """out = x + f(x), f(h) = experts(h) + down(gelu(up(h))), the experts chosen by
    a router; or, with norms,

        out = alpha x + sigmoid(gate . h) * norm(f(h)) . post,   h = norm(x) . pre

    Wr [E, d] are the router's weights and ``layer`` a binding.MoeLayer over
    the E experts; ``up`` [h, d] and ``down`` [d, h] the dense expert, or None:
    bfloat16, or both in MXFP4 (binding.quantize_rows_mxfp4), whose rows then are
    too.  ``pre`` and ``post`` are fp32 [d] weights of the norms (binding.block_norm;
    post None: f is not normalised), ``gate`` bfloat16 [1, d] or None (no gate);
    post, gate and an ``alpha`` of not 1 come with ``pre``.  ``score``, ``norm``,
    ``scale`` and the per-expert selection ``bias`` are moe_route's."""

    def __init__(self, layer: B.MoeLayer, Wr, k: int, up=None, down=None, bias=None,
                 score: str = "softmax", norm: bool = True, scale: float = 1.0, pre=None,
                 post=None, gate=None, alpha: float = 1.0, eps: float = 1e-6):
        if pre is None and (post is not None or gate is not None or alpha != 1.0):
            raise ValueError("post, gate and alpha come with pre")
        if isinstance(up, B.Mxfp4Rows) != isinstance(down, B.Mxfp4Rows):
            raise ValueError("the dense expert is in MXFP4 as a whole or not at all")
        self.layer, self.Wr, self.k = layer, Wr, k
        self.up, self.down, self.bias = up, down, bias
        self.pre, self.post, self.gate, self.alpha, self.eps = pre, post, gate, alpha, eps
        self.how = dict(score=score, norm=norm, scale=scale)
        self._master = None

    def route(self, x, mask=None, stats: bool = False) -> dict:
        """The router alone: its fp32 logits and what ``binding.route`` returns."""
        logits = B.linear(x, self.Wr, out_dtype=torch.float32)
        r = B.route(logits, self.k, bias=self.bias, mask=mask, stats=stats, **self.how)
        r["logits"] = logits
        return r

    def status(self) -> int:
        """Status bits (binding.STATUS_*) of the routed layer's last call and of
        what the device's router and dense products reported since this was
        last asked (binding.take_status); waits for the current stream."""
        bits = B.take_status(self.Wr.device)
        if self.layer is not None and self.layer._ws is not None:
            bits |= B.read_status(self.layer._ws)
        return bits

    def _dense(self, h, rows, y):
        """y + down(gelu(up(h))), into y; ``rows``: h, or its MXFP4 rows."""
        if isinstance(self.up, B.Mxfp4Rows):
            hid = B.linear_mxfp4(rows, self.up, act="gelu_tanh")
            return B.linear_mxfp4(hid, self.down, residual=y, y=y)
        return B.linear(B.linear(h, self.up, act="gelu_tanh"), self.down, residual=y, y=y)

    def _before(self) -> dict:
        """What block_norm takes of the norm before this block."""
        return dict(pre=self.pre, eps=self.eps, mxfp4=isinstance(self.up, B.Mxfp4Rows))

    def _inside(self, n: dict, mask):
        """f(h) and the tokens' gates, of what block_norm returned."""
        h = n["h"]
        r = self.route(h, mask)
        y = self.layer.forward(h, r["ids"], r["w"])
        if self.up is not None:
            y = self._dense(h, n.get("mx", h), y)
        if self.gate is None:
            return y, None
        return y, B.linear(h, self.gate, out_dtype=torch.float32).view(-1)

    def _after(self, o, g) -> dict:
        """What block_norm takes of the norm, gate and residual after this block."""
        return dict(o=o, post=self.post, post_norm=self.post is not None, gate=g,
                    gate_act="sigmoid", alpha=self.alpha, eps=self.eps)

    def forward(self, x, mask=None):
        """x [T, d] to [T, d], bf16 (with norms, or float32); rows with mask 0 are
        routed nowhere (with norms they are not read, and come out as 0)."""
        if self.pre is not None:
            return run_blocks([self], x, mask)
        if x.dtype != torch.bfloat16:
            raise ValueError(f"x: the routed experts take bfloat16, got {x.dtype}")
        r = self.route(x, mask)
        y = self.layer.forward(x, r["ids"], r["w"])
        # the residual stream rides on the dense expert's down projection, or
        # is added to the experts' sum as it is
        y.add_(x)
        return y if self.up is None else self._dense(x, x, y)

    def train_router(self, x, lr: float, balance: float = 1e-2, z: float = 1e-3, dw=None,
                     mask=None, grad_scale: float = 1.0):
        """One SGD step on Wr for balance * (balance loss) + z * (z loss) (and,
        with ``dw`` [T, k], the loss whose gradient with respect to the
        routing weights it is).  Returns (losses [2], dx): the losses before
        the step and the gradient with respect to x, times ``grad_scale`` (what
        a 16-bit dx cannot hold otherwise; dx is 0 where mask is).

        With norms x is the residual stream, and dx goes through the norm before
        the router (whose weights stay as they are).

        Wr holds the 16-bit values of weights kept in fp32, so that steps
        smaller than its spacing add up; entries of Wr that were set since the
        last step start from what they were set to."""
        stream = x
        if self.pre is not None:
            x = B.block_norm(x, pre=self.pre, mask=mask, eps=self.eps, h_dtype=self.Wr.dtype)["h"]
        elif mask is not None:
            # such a row may hold anything, and 0 times a NaN is one
            x = torch.where(mask.bool()[:, None], x, 0.0)
        r = self.route(x, mask, stats=True)
        dloss = torch.empty(2, dtype=torch.float32, device=x.device)
        dloss[0].fill_(balance * grad_scale)
        dloss[1].fill_(z * grad_scale)
        if dw is not None and grad_scale != 1.0:
            dw = dw * grad_scale
        dlogits = B.route_grad(r["logits"], r["ids"], r["counts"], dw=dw, dloss=dloss, mask=mask,
                               **self.how)
        dx, dWr, _ = B.linear_grad(x, self.Wr, dlogits, need=(True, True, False),
                                   dw_dtype=torch.float32)
        W, w = self.Wr, self._master
        if w is None or w.shape != W.shape or w.device != W.device:
            w = W.float()
        else:
            w = torch.where(w.to(W.dtype) == W, w, W.float())
        w.sub_(dWr, alpha=lr / grad_scale)
        W.copy_(w)
        self._master = w
        if self.pre is not None:
            dx = B.block_norm_grad(stream, dh=dx, pre=self.pre, mask=mask, eps=self.eps,
                                   weights=False)["dx"]
        return r["loss"], dx


def run_blocks(blocks, x, mask=None):
    """x [T, d] through blocks with norms, one after another: the norm after a
    block, its gate, the residual and the norm before the next block are one pass.
    x is bfloat16 or float32 and is left as it is; mask as in MoeBlock.forward."""
    blocks = list(blocks)
    if any(b.pre is None for b in blocks) or len({b.eps for b in blocks}) > 1:
        raise ValueError("blocks: all with norms, and of one eps")
    if x.dtype not in (torch.bfloat16, torch.float32):
        raise ValueError(f"x: bfloat16 or float32, got {x.dtype}")
    n = own = None  # own: the stream's buffer once it is not the caller's
    for b in blocks:
        if n is None:
            n = B.block_norm(x, mask=mask, h_dtype=torch.bfloat16, **b._before())
        else:
            n = B.block_norm(x, mask=mask, xn=own, **{**last, **b._before()})
            x = own = n["xn"]
        last = b._after(*b._inside(n, mask))
    return x if n is None else B.block_norm(x, mask=mask, xn=own, **last)["xn"]


def main():
    torch.manual_seed(0)
    T, d, E, k, f, h = 512, 256, 32, 4, 128, 512
    dev, bf = "cuda", torch.bfloat16

    def randn(*shape, amp=1.0):
        return (amp * torch.randn(*shape, device=dev)).to(bf)

    layer = B.MoeLayer(randn(E, d, f, amp=0.05), randn(E, d, f, amp=0.05),
                       randn(E, f, d, amp=0.05))
    # a router that prefers some experts
    Wr = randn(E, d, amp=0.03) + randn(E, 1, amp=0.02)
    block = MoeBlock(layer, Wr, k, up=randn(h, d, amp=0.05), down=randn(d, h, amp=0.05))
    x = randn(T, d) + 0.3
    print("block output", tuple(block.forward(x).shape))
    for step in range(60):
        loss, _ = block.train_router(x, lr=0.05, balance=1.0, z=1e-2)
        if step % 10 == 0 or step == 59:
            counts = block.route(x, stats=True)["counts"][:E]
            print(f"step {step:2d}: balance loss {float(loss[0]):.4f}  z loss {float(loss[1]):.3f}"
                  f"  tokens of the busiest expert {int(counts.max())} (mean {T * k // E})")
    # three blocks in a row: norms, a gate, the dense expert in MXFP4
    norm = torch.rand(d, device=dev) + 0.5
    dense = dict(up=B.quantize_rows_mxfp4(block.up), down=B.quantize_rows_mxfp4(block.down))
    normed = MoeBlock(layer, Wr, k, **dense, pre=norm, post=norm, gate=randn(1, d, amp=0.1))
    print("three blocks with norms", tuple(run_blocks([normed] * 3, x).shape))
    print("status bits", block.status())


if __name__ == "__main__":
    main()
