"""The logit of a row's target is formed in FP32, apart from the tensor cores' sums, in both directions of the cross entropy."""

import math

import pytest
import torch

from test_gpu_linear_ce import error_bits
from test_gpu_linear_ce_precision import confident, truncated_logit

pytestmark = pytest.mark.gpu

E24 = 2.0 ** -24


@pytest.mark.parametrize("T,calls", [(1, 256), (64, 8), (65, 8), (512, 2), (1500, 1)])
@pytest.mark.parametrize("D", [512, 1024, 2048, 7168])
def test_no_loss_is_too_large_for_what_the_tensor_cores_cut_off(T, calls, D):
    """Cutting off makes lse too small, where the logits that carry it are positive, but no longer the target's logit:
    losses are low, never high but for roundings.  Those of lse (in [8, 16): its sum in base 2, its product with ln 2)
    and of a target's logit near 10 (products of 8 elements and a tree: fewer than 16 roundings) have a deviation below
    16 2^-21 / sqrt(12) a token; the mean over the tokens is six of its deviations off at most."""
    from mixture_experts_routed_route_gb300 import loss
    V = 3000
    g = torch.Generator(device="cuda").manual_seed(D + T)
    weight = (2.0 * D ** -0.5 * torch.randn((V, D), generator=g, device="cuda")).bfloat16()
    w64 = weight.double()
    errors, most = [], []
    for _ in range(calls):
        targets = torch.randint(0, V, (T,), generator=g, device="cuda")
        h = (torch.randn((T, D), generator=g, device="cuda") + 2.5 * weight[targets].float()).bfloat16()
        value, _ = loss.linear_cross_entropy(h, weight, targets)
        logits = h.double() @ w64.t()
        ref = torch.logsumexp(logits, 1) - logits.gather(1, targets[:, None])[:, 0]
        errors.append(value.double() - ref)
        # a step of 16 elements cuts off at most 2^-23 of what its sum holds
        most.append((32 if D <= 1024 else 64) * 2 * E24 * float((h.double().abs() @ w64.abs().t()).max()))
    errors = torch.cat(errors)
    noise = 6 * 16 * 2.0 ** -21 / 12 ** 0.5 / errors.numel() ** 0.5
    print(T, D, "mean", float(errors.mean()), "noise", noise)
    assert float(errors.mean()) <= noise and float(errors.mean()) >= -max(most) - noise
    assert error_bits() == 0


@pytest.mark.parametrize("T", [3, 64, 65, 1100])
@pytest.mark.parametrize("D,V", [(7168, 1300), (1024, 1200), (264, 1200)])
def test_confident_tokens_of_any_lse(T, D, V):
    """Probabilities around 0.9997 at a logit near 40: the loss and the gradient, from the forward's lse and from one in 64
    bits, are as good as FP32 makes them.  The target's logit goes through fewer than 32 roundings (eight products in a
    row, up to four rows of them a thread, a tree), of at most half a step of 64 each; the others' error is a share of
    themselves."""
    from mixture_experts_routed_route_gb300 import loss
    h, weight, targets = confident(T, D, V, 40.0, 40.0 - 8.1 - math.log(V), T + D)
    h64, w64 = h.double(), weight.double()
    logits = h64 @ w64.t()
    hit = logits.gather(1, targets[:, None])[:, 0]
    lse = torch.logsumexp(logits, 1)
    rows = torch.arange(T, device="cuda")
    p = torch.exp(logits - lse[:, None])
    left = 1 - p[rows, targets]
    value, mine = loss.linear_cross_entropy(h, weight, targets)
    # independent roundings of that number: six of their deviations, 2^-18 / sqrt(12) each, whose values grow to 40
    dot = 6 * 32 ** 0.5 * 2.0 ** -18 / 12 ** 0.5
    # a logit near 25 in sums of up to 1024 elements
    others = float(truncated_logit(h64, w64[(targets + 1) % V], 64).max())
    # log2 of a sum near 1 and the parts' joining: a few steps of 1
    assert bool(((value.double() - (lse - hit)).abs() <= left * (others + dot) + 2.0 ** -20).all())
    d = torch.full((T,), 1.0 / T, device="cuda")
    g = (p - torch.zeros_like(p).scatter_(1, targets[:, None], 1.0)) * d.double()[:, None]
    one_sum = float(truncated_logit(h64, w64[(targets + 1) % V], 1 << 20).max())
    # lse in FP32 and its product with log2 e, the exponential, as in test_gpu_linear_ce_precision.py
    scale = 2.0 ** -19 * (1 + math.log(2)) + 2.0 ** -21
    for ls, own in ((lse.float(), 0.0), (mine, 2.0 ** -19 * (1 + 2 * math.log(2)) + 2.0 ** -20)):
        dh, dw = loss.linear_cross_entropy_backward(h, weight, targets, ls, d)
        rel = (scale + own + dot) * p[rows, targets] / left + one_sum + others + 2.0 ** -8
        for got, ref, mag in ((dh, g @ w64, g.abs() @ w64.abs()), (dw[targets], (g.t() @ h64)[targets], (g.abs().t() @ h64.abs())[targets])):
            err = (got.double() - ref).norm(dim=1)
            print(T, D, "off", float((err / ref.norm(dim=1)).max()), "of", float((err / (rel * mag.norm(dim=1) + 2.0 ** -8 * ref.norm(dim=1))).max()))
            assert bool((err <= rel * mag.norm(dim=1) + 2.0 ** -8 * ref.norm(dim=1)).all())
    assert error_bits() == 0
