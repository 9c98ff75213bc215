"""Workspaces of the cross entropy: one made for T tokens takes every call on fewer."""

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T,D,V", [(300, 64, 1000), (256, 256, 32768), (1, 8, 7), (64, 72, 300), (1500, 16, 129)])
def test_a_workspace_for_more_tokens(T, D, V):
    from mixture_experts_routed_route_gb300 import loss, optim
    g = torch.Generator(device="cuda").manual_seed(T)
    weight = (2.0 * D ** -0.5 * torch.randn((V, D), generator=g, device="cuda")).bfloat16()
    h = torch.randn((T, D), generator=g, device="cuda").bfloat16()
    targets = torch.randint(0, V, (T,), generator=g, device="cuda")
    fw, bw = loss.workspace(T, D, V, backward=False), loss.workspace(T, D, V)
    for n in sorted({0, 1, 2, 63, 64, 65, 255, 256, 257, T - 1, T}):
        if n > T:
            continue
        d = torch.full((n,), 0.5, device="cuda")
        want = loss.linear_cross_entropy(h[:n], weight, targets[:n])
        got = loss.linear_cross_entropy(h[:n], weight, targets[:n], workspace=fw)
        assert all(torch.equal(a, b) for a, b in zip(got, want)), n
        loss.linear_cross_entropy_backward(h[:n], weight, targets[:n], want[1], d, workspace=bw)
    assert optim.error_bits() == 0
