"""How far the cross entropy's gradients are off, against 64 bits."""

import math

import pytest
import torch

pytestmark = pytest.mark.gpu

E24 = 2.0 ** -24


def confident(T, D, V, top, rest, seed):
    """Rows whose target's logit is near `top` and whose other logits are near `rest`: products along two unit
    directions that h and the weights share, so that a logit's partial sums grow steadily."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda", dtype=torch.float64)  # noqa: E731
    u = r(D)
    u /= u.norm()
    n = r(V, D)
    n /= n.norm(dim=1, keepdim=True)
    targets = torch.randperm(V, generator=g, device="cuda")[:T]
    a, b = rest ** 0.5, (top - rest) ** 0.5
    weight = (a * u + b * n).bfloat16()
    h = (a * u + b * n[targets]).bfloat16()
    return h, weight, targets


def truncated_logit(h, w, steps):
    """What a logit of the products h w may be off by where every 16 of them join a sum that cuts off at 2^-23 of
    itself, by at most one such width a step, in sums of `steps` that are joined in 32 bits: a rounding (2^-24 of the
    running sum) for each."""
    T, D = h.shape
    p = torch.nn.functional.pad(h * w, (0, -D % 16)).view(T, -1, 16).sum(2)
    off, total = 0.0, 0.0
    for k in range(0, p.shape[1], steps):
        off = off + 2 * E24 * p[:, k:k + steps].cumsum(1).abs().sum(1)
        total = total + p[:, k:k + steps].sum(1)
        off = off + E24 * total.abs()
    return off


@pytest.mark.parametrize("T", [3, 64, 65, 200])
@pytest.mark.parametrize("D,V", [(7168, 1000), (1408, 700), (4104, 1100)])
def test_confident_tokens(T, D, V):
    """Tokens of probabilities around 0.9997 at a logit near 40: a gradient is a difference of nearly equal numbers, and is off
    by what the logit is off by.  With lse from 64 bits that is what cutting off in sums of 1024 elements loses; with
    the forward's own, the two products' logits are off alike, and the loss of bits is lse's alone."""
    from mixture_experts_routed_route_gb300 import loss, optim
    top = 40.0
    rest = top - 8.1 - math.log(V)
    h, weight, targets = confident(T, D, V, top, rest, T + D)
    h64, w64 = h.double(), weight.double()
    logits = h64 @ w64.t()
    hit = logits.gather(1, targets[:, None])[:, 0]
    lse = torch.logsumexp(logits, 1)
    rows = torch.arange(T, device="cuda")
    p = torch.exp(logits - lse[:, None])
    left = 1 - p[rows, targets]
    assert float(left.min()) > 1e-5 and float(left.max()) < 1e-2 and 35 < float(hit.min()) and float(hit.max()) < 45
    d = torch.full((T,), 1.0 / T, device="cuda")
    g = (p - torch.zeros_like(p).scatter_(1, targets[:, None], 1.0)) * d.double()[:, None]
    # lse in FP32 and its product with log2 e: half a step of 40 and of 58 (2^-19, of log2 that times ln 2); exp2's
    # argument below 16 to 2^-21 where it counts, the exponential's own 2^-22
    scale = 2.0 ** -19 * (1 + math.log(2)) + 2.0 ** -21
    off = truncated_logit(h64, w64[targets], 64) + scale
    # the forward's lse: its sum, logarithm and product with ln 2 lose a half step of 58 twice more
    own = 2 * scale + 2.0 ** -19 * 2 * math.log(2) + 2.0 ** -20
    _, mine = loss.linear_cross_entropy(h, weight, targets)
    for ls, lost in ((lse.float(), off), (mine, torch.full_like(off, own))):
        dh, dw = loss.linear_cross_entropy_backward(h, weight, targets, ls, d)
        # Relative to each g: the target's logit error as a share of what is left of 1; 2^-12 covers the others' own logit
        # errors (25 times 1e-6) and what all share; g's rounding 2^-8, the result's 2^-8.
        rel = lost * p[rows, targets] / left
        ref, mag = g @ w64, g.abs() @ w64.abs()
        tol = (rel + 2.0 ** -12 + 2.0 ** -8) * mag.norm(dim=1) + 2.0 ** -8 * ref.norm(dim=1)
        err = (dh.double() - ref).norm(dim=1)
        print(T, D, V, "off", float((err / ref.norm(dim=1)).max()), "of", float((err / tol).max()))
        assert bool((err <= tol).all())
        ref, mag = (g.t() @ h64)[targets], (g.abs().t() @ h64.abs())[targets]
        tol = (rel + 2.0 ** -12 + 2.0 ** -8) * mag.norm(dim=1) + 2.0 ** -8 * ref.norm(dim=1)
        err = (dw[targets].double() - ref).norm(dim=1)
        print(T, D, V, "off", float((err / ref.norm(dim=1)).max()), "of", float((err / tol).max()))
        assert bool((err <= tol).all())
    assert optim.error_bits() == 0
