"""The token example: embedding, norms with dropout, router, experts, head and
loss, their backward and the update run together, and what they give is the
gradient of the loss."""

import os
import sys

import pytest
import torch

import dropout_oracle as oracle

pytestmark = pytest.mark.gpu

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


def plain_loss(p, tokens, targets, ids, keep):
    """The mean loss in 64 bits, no rounding in between, at given expert ids and dropout mask."""
    def norm(t, w, b):
        d = t - t.mean(1, keepdim=True)
        return d * ((d * d).mean(1, keepdim=True) + 1e-5) ** -0.5 * w + b

    x = p["embed"][tokens]
    h = norm(x, p["w1"], p["b1"])
    scores = torch.softmax(torch.gather(h @ p["router"], 1, ids), 1)
    w13, wo = p["w13"][ids], p["wo"][ids]
    F = wo.shape[-1]
    h1 = torch.einsum("tkfd,td->tkf", w13, h)
    h2 = torch.nn.functional.silu(h1[..., :F]) * h1[..., F:]
    o = torch.einsum("tk,tkdf,tkf->td", scores, wo, h2)
    u = norm(x + o * keep, p["w2"], p["b2"])
    logits = u @ p["head"].t()
    on = targets >= 0
    return (torch.logsumexp(logits[on], 1) - logits[on].gather(1, targets[on][:, None])[:, 0]).mean()


def test_gradients_of_the_whole_model():
    import train_tokens
    m = train_tokens.Model(T=48, V=300, D=128, F=128, E=4, K=2, p=0.25, seed=3)
    tokens, targets = train_tokens.batch(m)
    counted = int((targets >= 0).sum())
    value = m.forward(tokens, targets)
    grads = m.backward(torch.full((48,), 1.0 / counted, device="cuda"))
    k, f = oracle.keep(48, 128, 0.25, 3 + 12345, 0, 1)
    names = ("embed", "w1", "b1", "w2", "b2", "router", "w13", "wo", "head")
    p = {n: (m.head16 if n == "head" else getattr(m, n)).double().requires_grad_(True) for n in names}
    ref = plain_loss(p, tokens, targets, m.ids.long(), k.cuda().double() * f)
    # the logits are of sixteen-bit rows: a loss near 6 moves by a few of their roundings
    at = float(ref.detach())
    assert abs(float(value.sum()) / counted - at) <= 4 * 2.0 ** -9 * at
    want = torch.autograd.grad(ref, [p[n] for n in names])
    # experts, norms' results and the logits' gradient are BF16: about sixteen roundings of 2^-9 (in norm) there and back
    for n, r in zip(names, want):
        assert float((grads[n].double() - r).norm() / r.norm()) <= 16 * 2.0 ** -9, n
    m.layer.close()


def test_a_few_steps_run():
    import train_tokens
    losses = train_tokens.train(steps=4)
    assert all(v == v and abs(v) < 1e4 for v in losses)
