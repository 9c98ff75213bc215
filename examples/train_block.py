"""A few training steps of one transformer block's feed-forward half, on one GPU:

    h = rms_norm(x) * pre_weight                      block.block_norm
    ids, scores = top_k of h @ router                 block.topk_gate
    o = routed experts of h                           layer.MoELayer (BF16)
    y = x + gate * rms_norm(o) * post_weight          block.block_norm
    loss = mean (y - target)^2 / 2

and back: the block norm's gradients, the experts' (with the score gradient),
the router's, the first norm's; then a Muon step on the stacked expert weights
(optim.Muon: W13 as 2E matrices, gate and up apart) and plain gradient steps on
the rest.  The residual stream is FP32, everything the experts see is BF16.

    python examples/train_block.py [--steps 20]
"""

import argparse
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch

from mixture_experts_routed_route_gb300 import block, optim
from mixture_experts_routed_route_gb300.layer import MoELayer, PreparedWeight


class Block:
    """The parameters of one block, its forward, backward and update."""

    def __init__(self, T=128, D=256, F=512, E=8, K=2, device="cuda", seed=0, lr=2e-2):
        g = torch.Generator(device=device)
        g.manual_seed(seed)
        rnd = lambda *s: torch.randn(s, generator=g, device=device)  # noqa: E731
        self.T, self.D, self.F, self.E, self.K = T, D, F, E, K
        self.device = torch.device(device)
        self.pre_weight = torch.ones(D, device=device)
        self.post_weight = torch.ones(D, device=device)
        self.gate = torch.full((D,), 0.5, device=device)
        self.router = rnd(D, E) * D ** -0.5
        self.w13 = (rnd(E, 2 * F, D) * D ** -0.5).bfloat16()
        self.w2 = (rnd(E, D, F) * F ** -0.5).bfloat16()
        self.layer = MoELayer(T, D, F, E, K, "bf16", training=True, device=device)
        self.saved = self.layer.new_saved()
        self.muon = optim.Muon([self.w13.view(2 * E, F, D), self.w2], lr=lr, master=True)
        self.lr = lr
        self.prepare()

    def prepare(self):
        """The experts' weights as the layer reads them (again after each update)."""
        self.W13 = PreparedWeight(self.w13, "bf16")
        self.W2 = PreparedWeight(self.w2, "bf16")

    def forward(self, x):
        """y [T, D] of x (float32); keeps what the backward needs."""
        T, dev = x.shape[0], x.device
        self.x = x
        self.pre_stats = torch.empty((2, T), device=dev)
        self.post_stats = torch.empty((2, T), device=dev)
        _, self.h = block.block_norm(x, pre_weight=self.pre_weight, stats=self.pre_stats)
        self.logits = self.h.float() @ self.router
        self.ids, self.scores = block.topk_gate(self.logits, self.K, renormalize=True)
        self.o = self.layer.forward(self.h, self.ids, self.scores, self.W13, self.W2, saved=self.saved)
        y, _ = block.block_norm(x, self.o, gate=self.gate, post_weight=self.post_weight, stats=self.post_stats)
        return y

    def backward(self, dy):
        """Gradients of x and of every parameter, by name."""
        post = block.block_norm_backward(self.x, self.o, self.post_stats, dy, gate=self.gate,
                                         post_weight=self.post_weight)
        d_scores = torch.empty_like(self.scores)
        dh, dw13, dw2 = self.layer.backward(self.saved, post.dbranch, self.W13, self.W2, d_scores=d_scores)
        d_logits = block.topk_gate_backward(self.logits, self.ids, d_scores, renormalize=True)
        dh = (dh.float() + d_logits @ self.router.t()).bfloat16()
        pre = block.block_norm_backward(self.x, None, self.pre_stats, post.dx, dh, pre_weight=self.pre_weight)
        return {"x": pre.dx, "pre_weight": pre.dpre_weight, "post_weight": post.dpost_weight, "gate": post.dgate,
                "router": self.h.float().t() @ d_logits, "w13": dw13, "w2": dw2}

    def update(self, grads):
        self.muon.step([grads["w13"].view(2 * self.E, self.F, self.D), grads["w2"]])
        self.prepare()
        for name in ("pre_weight", "post_weight", "gate", "router"):
            getattr(self, name).sub_(self.lr * grads[name])


def train(steps=20, seed=0, **shape):
    """Losses of `steps` steps towards a fixed target."""
    b = Block(seed=seed, **shape)
    g = torch.Generator(device=b.device)
    g.manual_seed(seed + 1)
    x = torch.randn((b.T, b.D), generator=g, device=b.device)
    target = x + 0.5 * torch.randn((b.T, b.D), generator=g, device=b.device)
    losses = []
    for _ in range(steps):
        diff = b.forward(x) - target
        losses.append(0.5 * diff.square().mean())
        b.update(b.backward(diff / diff.numel() * b.T))   # the loss of a token's mean, so that steps do not shrink with T
    losses = [float(v) for v in losses]
    bits = b.layer.error_bits() | optim.error_bits(b.device)
    b.layer.close()
    if bits:
        raise RuntimeError(f"device error bits {bits:#x}")
    return losses


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--steps", type=int, default=20)
    for i, loss in enumerate(train(ap.parse_args().steps)):
        print(f"step {i:3d}  loss {loss:.5f}")
