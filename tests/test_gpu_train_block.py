"""The block example: norm, router, experts, gate and residual, their backward
and the Muon update run together, and what they give is the gradient of the
block's loss."""

import os
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


def plain_loss(p, x, target, ids):
    """The block's loss in 64 bits, no rounding in between, at given expert ids."""
    def norm(t, w):
        return t * ((t * t).mean(1, keepdim=True) + 1e-6) ** -0.5 * w

    h = norm(x, p["pre_weight"])
    scores = torch.softmax(torch.gather(h @ p["router"], 1, ids), 1)
    w13, w2 = p["w13"][ids], p["w2"][ids]
    F = w2.shape[-1]
    h1 = torch.einsum("tkfd,td->tkf", w13, h)
    h2 = torch.nn.functional.silu(h1[..., :F]) * h1[..., F:]
    o = torch.einsum("tk,tkdf,tkf->td", scores, w2, h2)
    y = x + p["gate"] * norm(o, p["post_weight"])
    return 0.5 * (y - target).square().mean()


def test_gradients_of_the_whole_block():
    import train_block
    b = train_block.Block(T=32, D=128, F=128, E=4, K=2, seed=3)
    x = torch.randn((32, 128), device="cuda", generator=torch.Generator("cuda").manual_seed(1))
    target = torch.randn((32, 128), device="cuda", generator=torch.Generator("cuda").manual_seed(2))
    y = b.forward(x)
    grads = b.backward((y - target) / y.numel())
    names = ("pre_weight", "post_weight", "gate", "router", "w13", "w2")
    p = {n: getattr(b, n).double().requires_grad_(True) for n in names}
    x64 = x.double().requires_grad_(True)
    ref = torch.autograd.grad(plain_loss(p, x64, target.double(), b.ids.long()), [x64] + [p[n] for n in names])
    # the experts run in BF16: about a dozen roundings of 2^-9 (2e-3) on the way there and back, in norm
    for n, r in zip(("x",) + names, ref):
        assert float((grads[n].double() - r).norm() / r.norm()) <= 12 * 2.0 ** -9, n
    b.layer.close()


def test_training_lowers_the_loss():
    import train_block
    losses = train_block.train(steps=12, seed=0)
    assert all(v == v for v in losses)
    assert losses[-1] < 0.9 * losses[0]
