"""A few training steps of a small next-token model with one routed block, on one GPU:

    x = embed[tokens]
    h = layer_norm(x)                                    block.layer_norm
    ids, scores = top_k of h @ router                    block.topk_gate
    o = routed experts of h                              layer.MoELayer (BF16)
    y = x + dropout(o);  u = layer_norm(y)               block.layer_norm, one pass
    loss = mean cross entropy of u @ head.T              loss.linear_cross_entropy

and back: the head's and the loss's gradients without the logits in memory, both
norms' with dropout's mask drawn again, the experts', the router's; then a Muon
step on the stacked expert weights and plain gradient steps on the rest.  The
first tokens of each sequence are a prompt that takes no loss.

    python examples/train_tokens.py [--steps 20]
"""

import argparse
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch

from mixture_experts_routed_route_gb300 import block, loss, optim
from mixture_experts_routed_route_gb300.layer import MoELayer, PreparedWeight

IGNORE = -100


class Model:
    """The parameters of the model, its forward, backward and update."""

    def __init__(self, T=256, V=2000, D=256, F=256, E=8, K=2, p=0.1, device="cuda", seed=0, lr=2e-2):
        g = torch.Generator(device=device)
        g.manual_seed(seed)
        rnd = lambda *s: torch.randn(s, generator=g, device=device)  # noqa: E731
        self.T, self.V, self.D, self.F, self.E, self.K, self.p = T, V, D, F, E, K, p
        self.device = torch.device(device)
        self.embed = rnd(V, D)
        self.w1, self.b1 = torch.ones(D, device=device), torch.zeros(D, device=device)
        self.w2, self.b2 = torch.ones(D, device=device), torch.zeros(D, device=device)
        self.router = rnd(D, E) * D ** -0.5
        self.w13 = (rnd(E, 2 * F, D) * D ** -0.5).bfloat16()
        self.wo = (rnd(E, D, F) * F ** -0.5).bfloat16()
        self.head = rnd(V, D) * D ** -0.5
        self.rng = torch.tensor([seed + 12345, 0], dtype=torch.int64, device=device)   # dropout's seed and step
        self.layer = MoELayer(T, D, F, E, K, "bf16", training=True, device=device)
        self.saved = self.layer.new_saved()
        self.muon = optim.Muon([self.w13.view(2 * E, F, D), self.wo], lr=lr, master=True)
        self.lr = lr
        self.prepare()

    def prepare(self):
        """The weights as the products read them (again after each update)."""
        self.W13 = PreparedWeight(self.w13, "bf16")
        self.Wo = PreparedWeight(self.wo, "bf16")
        self.head16 = self.head.bfloat16()

    def forward(self, tokens, targets):
        """Each token's loss (0 where its target is ignored); keeps what the backward needs."""
        T, dev = tokens.shape[0], tokens.device
        self.tokens, self.targets = tokens, targets
        self.x = self.embed[tokens]
        self.stats1, self.stats2 = torch.empty((2, T), device=dev), torch.empty((2, T), device=dev)
        _, self.h = block.layer_norm(self.x, weight=self.w1, bias=self.b1, stats=self.stats1)
        self.logits = self.h.float() @ self.router
        self.ids, self.scores = block.topk_gate(self.logits, self.K, renormalize=True)
        o = self.layer.forward(self.h, self.ids, self.scores, self.W13, self.Wo, saved=self.saved)
        self.y, self.u = block.layer_norm(self.x, o, weight=self.w2, bias=self.b2, dropout=self.p, rng=self.rng, site=1,
                                          stats=self.stats2)
        value, self.lse = loss.linear_cross_entropy(self.u, self.head16, targets, ignore_index=IGNORE)
        return value

    def backward(self, d_loss):
        """Gradients of every parameter, by name, from that of each token's loss."""
        du, dhead = loss.linear_cross_entropy_backward(self.u, self.head16, self.targets, self.lse, d_loss,
                                                       ignore_index=IGNORE)
        post = block.layer_norm_backward(self.y, self.stats2, du, weight=self.w2, bias=self.b2, dropout=self.p,
                                         rng=self.rng, site=1)
        d_scores = torch.empty_like(self.scores)
        dh, dw13, dwo = self.layer.backward(self.saved, post.dbranch, self.W13, self.Wo, d_scores=d_scores)
        d_logits = block.topk_gate_backward(self.logits, self.ids, d_scores, renormalize=True)
        dh = (dh.float() + d_logits @ self.router.t()).bfloat16()
        pre = block.layer_norm_backward(self.x, self.stats1, dh, post.dx, weight=self.w1, bias=self.b1, branch=False)
        embed = torch.zeros_like(self.embed).index_add_(0, self.tokens, pre.dx)
        return {"embed": embed, "w1": pre.dweight, "b1": pre.dbias, "w2": post.dweight, "b2": post.dbias,
                "router": self.h.float().t() @ d_logits, "w13": dw13, "wo": dwo, "head": dhead}

    def update(self, grads):
        self.muon.step([grads["w13"].view(2 * self.E, self.F, self.D), grads["wo"]])
        for name in ("embed", "w1", "b1", "w2", "b2", "router", "head"):
            getattr(self, name).sub_(self.lr * grads[name])
        self.rng[1] += 1
        self.prepare()


def batch(m, seed=1, prompt=0.25):
    """Tokens and their targets: a fixed successor of each token, the first ones ignored."""
    g = torch.Generator(device=m.device)
    g.manual_seed(seed)
    tokens = torch.randint(0, m.V, (m.T,), generator=g, device=m.device)
    targets = (tokens * 7 + 3) % m.V
    targets[:int(prompt * m.T)] = IGNORE
    return tokens, targets


def train(steps=20, seed=0, **shape):
    """Mean losses of `steps` steps on one batch."""
    m = Model(seed=seed, **shape)
    tokens, targets = batch(m)
    counted = (targets != IGNORE).sum()
    d_loss = torch.ones(m.T, device=m.device) / counted
    losses = []
    for _ in range(steps):
        losses.append(m.forward(tokens, targets).sum() / counted)
        m.update(m.backward(d_loss))
    losses = [float(v) for v in losses]
    bits = m.layer.error_bits() | optim.error_bits(m.device)
    m.layer.close()
    if bits:
        raise RuntimeError(f"device error bits {bits:#x}")
    return losses


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--steps", type=int, default=20)
    for i, value in enumerate(train(ap.parse_args().steps)):
        print(f"step {i:3d}  loss {value:.5f}")
