"""A whole mixture-of-experts block on the library: router, routed experts, a
dense expert beside them and the residual; and a training step of the router.

    python -m moe_prefill_routing_gb300.block      # needs a GB300

``MoeBlock.forward`` is what a model runs per layer (a prefill chunk or a few
decoded tokens); ``MoeBlock.train_router`` takes one gradient step that
balances the experts, the experts' weights fixed.
"""
from __future__ import annotations

import torch

from . import binding as B


class MoeBlock:
    """out = x + experts(x) + down(gelu(up(x))), the experts chosen by a router.

    Wr [E, d] are the router's weights and ``layer`` a binding.MoeLayer over
    the E experts; ``up`` [h, d] and ``down`` [d, h] the dense expert, or None.
    ``score``, ``norm``, ``scale`` and the per-expert selection ``bias`` are
    moe_route's."""

    def __init__(self, layer: B.MoeLayer, Wr, k: int, up=None, down=None, bias=None,
                 score: str = "softmax", norm: bool = True, scale: float = 1.0):
        self.layer, self.Wr, self.k = layer, Wr, k
        self.up, self.down, self.bias = up, down, bias
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

    def forward(self, x, mask=None):
        """x [T, d] bf16 to [T, d]; rows with mask 0 are routed nowhere."""
        if x.dtype != torch.bfloat16:
            raise ValueError(f"x: the routed experts take bfloat16, got {x.dtype}")
        r = self.route(x, mask)
        y = self.layer.forward(x, r["ids"], r["w"])
        # the residual stream rides on the dense expert's down projection, or
        # is added to the experts' sum as it is
        if self.up is None:
            return y.add_(x)
        h = B.linear(x, self.up, act="gelu_tanh")
        return B.linear(h, self.down, residual=y.add_(x), y=y)

    def train_router(self, x, lr: float, balance: float = 1e-2, z: float = 1e-3, dw=None,
                     mask=None, grad_scale: float = 1.0):
        """One SGD step on Wr for balance * (balance loss) + z * (z loss) (and,
        with ``dw`` [T, k], the loss whose gradient with respect to the
        routing weights it is).  Returns (losses [2], dx): the losses before
        the step and the gradient with respect to x, times ``grad_scale`` (what
        a 16-bit dx cannot hold otherwise; dx is 0 where mask is).

        Wr holds the 16-bit values of weights kept in fp32, so that steps
        smaller than its spacing add up; entries of Wr that were set since the
        last step start from what they were set to."""
        if mask is not None:
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
        return r["loss"], dx


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
    print("status bits", block.status())


if __name__ == "__main__":
    main()
