"""A weight that all tokens share in the cross entropy's gradients, against 64 bits."""

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("N,weight_of", [(255, lambda n: 1.0 / n), (510, lambda n: 1.0 / n), (2040, lambda n: 1.0 / n),
                                         (300, lambda n: 0.7), (129, lambda n: -1.3e-20), (11, lambda n: 1.0 / 11)])
def test_a_weight_that_all_tokens_share(N, weight_of):
    """A mean's 1 / N is no rounding's business: g is rounded without it.  A result is then off by its own rounding (at
    most 2^-7 / sqrt(12) of itself in norm: uniform in a step) and by what the rounding of small probabilities and of
    p - 1 (at most p where p is below 2^-9) leaves: independent or tiny, no share of the whole."""
    from mixture_experts_routed_route_gb300 import loss, optim
    D, V = 256, 5000
    g = torch.Generator(device="cuda").manual_seed(N)
    weight = (0.25 * D ** -0.5 * torch.randn((V, D), generator=g, device="cuda")).bfloat16()
    h = torch.randn((N, D), generator=g, device="cuda").bfloat16()
    targets = torch.randint(0, V, (N,), generator=g, device="cuda")
    d = torch.full((N,), weight_of(N), device="cuda")
    logits = h.double() @ weight.double().t()
    lse = torch.logsumexp(logits, 1)
    p = torch.exp(logits - lse[:, None])
    assert float(p.max()) < 2.0 ** -9
    q = d.double()[:, None] * (p - torch.zeros_like(p).scatter_(1, targets[:, None], 1.0))
    dh, dw = loss.linear_cross_entropy_backward(h, weight, targets, lse.float(), d)
    for name, got, ref in (("dh", dh, q @ weight.double()), ("dweight", dw, q.t() @ h.double())):
        e = got.double() - ref
        norm, share = float(e.norm() / ref.norm()), float((e * ref).sum() / ref.norm() ** 2)
        print(N, name, "norm", norm, "share", share)
        assert norm <= 2.0 ** -7 / 12 ** 0.5 + float(p.max()), (name, norm)
        # independent roundings leave a share of 2^-8 over the root of their number, six deviations; p as above
        assert abs(share) <= float(p.max()) + 6 * 2.0 ** -8 * ref.numel() ** -0.5, (name, share)
    assert optim.error_bits() == 0


@pytest.mark.parametrize("T", [40, 300, 1500])
def test_weights_of_any_size_and_none(T):
    """An infinite or NaN weight spoils its own row of dh and no other; weights of zero alone give zeros; weights far
    apart keep each its own scale."""
    from mixture_experts_routed_route_gb300 import loss, optim
    D, V = 64, 700
    g = torch.Generator(device="cuda").manual_seed(T)
    weight = (D ** -0.5 * torch.randn((V, D), generator=g, device="cuda")).bfloat16()
    h = torch.randn((T, D), generator=g, device="cuda").bfloat16()
    targets = torch.randint(0, V, (T,), generator=g, device="cuda")
    _, lse = loss.linear_cross_entropy(h, weight, targets)
    back = lambda d: loss.linear_cross_entropy_backward(h, weight, targets, lse, d)  # noqa: E731
    d = torch.full((T,), 1.0 / T, device="cuda")
    want = back(d)[0]
    for bad in (float("inf"), float("-inf"), float("nan")):
        e = d.clone()
        e[T // 2] = bad
        dh = back(e)[0]
        keep = torch.arange(T, device="cuda") != T // 2
        assert torch.equal(dh[keep], want[keep]) and not bool(dh[T // 2].isfinite().any())
    dh, dw = back(torch.zeros_like(d))
    assert bool((dh == 0).all()) and bool((dw == 0).all())
    # powers of two beside the shared weight: every row's dh times that power, exactly
    power = 2.0 ** torch.randint(-60, 60, (T,), generator=g, device="cuda").float()
    assert torch.equal(back(d * power)[0].float(), want.float() * power[:, None])
    assert optim.error_bits() == 0
