"""The range of the orthogonalised updates: singular values up to the stated
limits on the way, schedules with steep polynomials, and zero matrices at any
eps, on the tiled and the small kernel, wide and tall.

Bounds.  Where every product is exact in the kernel's formats (powers of two
and small whole numbers) the result has to be the exact value rounded to
BF16.  Else as in test_gpu_muon.py."""

import pytest
import torch

from test_gpu_muon import BOUND, gradient, ns64, off

pytestmark = pytest.mark.gpu

# small kernel (wide, tall) and tiled kernels (wide, tall)
SHAPES = [(5, 96, 130), (5, 130, 96), (2, 300, 520), (2, 520, 300)]


def one_entry(E, N, K):
    """One nonzero entry a matrix, of several signs and sizes: its singular value starts at 1."""
    u = torch.zeros((E, N, K), device="cuda")
    for e in range(E):
        u[e, (7 * e) % N, (11 * e + 3) % K] = (-1.0) ** e * 2.0 ** (3 * e - 4)
    return u


@pytest.mark.parametrize("E,N,K", SHAPES)
@pytest.mark.parametrize("s", [6.0, 7.75, 11.0])
def test_singular_values_up_to_the_limit(E, N, K, s):
    """Steps that scale by s and by one: X s at the entry, A s^2 there."""
    from mixture_experts_routed_route_gb300 import optim
    u = one_entry(E, N, K)
    out = optim.orthogonalize(u, steps=2, coefficients=[(s, 0.0, 0.0), (1.0, 0.0, 0.0)], eps=1e-30)
    assert torch.equal(out, (s * u.sign()).bfloat16())
    assert optim.error_bits() == 0


@pytest.mark.parametrize("E,N,K", SHAPES)
@pytest.mark.parametrize("s", [6.0, 11.0])
def test_one_row_or_column(E, N, K, s):
    """A single row (wide) or column (tall): one large diagonal element of A."""
    from mixture_experts_routed_route_gb300 import optim
    u = torch.zeros((E, N, K), device="cuda")
    g = torch.Generator("cuda").manual_seed(3)
    if N <= K:
        u[:, 17] = torch.randn((E, K), generator=g, device="cuda")
    else:
        u[:, :, 17] = torch.randn((E, N), generator=g, device="cuda")
    table = [(s, 0.0, 0.0), (1.0, 0.0, 0.0)]
    assert off(optim.orthogonalize(u, steps=2, coefficients=table), ns64(u, 2, table)) <= BOUND


@pytest.mark.parametrize("E,N,K", SHAPES)
def test_polynomials_with_large_elements_off_the_diagonal(E, N, K):
    """Two equal rows (columns): A = 8 in a block of two, B = 15 A off its diagonal, X = (1 + 15 x 16) 4 in the end."""
    from mixture_experts_routed_route_gb300 import optim
    u = torch.zeros((E, N, K), device="cuda")
    u[:, 3:5, 8:10] = 1.0
    out = optim.orthogonalize(u, steps=2, coefficients=[(4.0, 0.0, 0.0), (1.0, 15.0, 0.0)], eps=1e-30)
    want = torch.zeros_like(u)
    want[:, 3:5, 8:10] = 0.5 * 4.0 * (1 + 15.0 * 16.0)
    assert torch.equal(out, want.bfloat16())


# 0 to 1 goes to 1.96 at most on the way, and to 1.12 at most in the end
STEEP = [(8.205, -22.902, 16.461), (4.066, -2.861, 0.518), (3.91, -2.823, 0.525), (3.286, -2.415, 0.485), (2.278, -1.62, 0.398)]


@pytest.mark.parametrize("E,N,K", SHAPES + [(3, 1000, 1531), (8, 512, 256)])
def test_schedule_with_a_steep_first_step(E, N, K):
    """Coefficients beyond 16 where the schedule keeps [0, 1] in range."""
    from mixture_experts_routed_route_gb300 import optim
    for u in (gradient(E, N, K, seed=4), torch.randn((E, N, K), device="cuda", generator=torch.Generator("cuda").manual_seed(5))):
        assert off(optim.orthogonalize(u, steps=5, coefficients=STEEP), ns64(u, 5, STEEP)) <= BOUND
    # a singular value at the end of [0, 1]: rounding X's hi half and A moves A by up to 3 x 2^-12 of itself and X by
    # that times s (b s^2 + 2 c s^4); with the slopes of the steps after it 0.006 from the second step (s = 1.76), 0.004
    # from the others, and the result's own rounding is 0.004
    u = one_entry(E, N, K)
    out = optim.orthogonalize(u, steps=5, coefficients=STEEP, eps=1e-30)
    assert float((out.double() - ns64(u, 5, STEEP, 1e-30)).abs().max()) <= 0.02
    assert optim.error_bits() == 0


@pytest.mark.parametrize("N,K", [(64, 96), (300, 280), (33, 7)])
@pytest.mark.parametrize("eps", [1e-7, 1e-36, 1e-38])
def test_zero_matrix_at_any_eps(N, K, eps):
    from mixture_experts_routed_route_gb300 import optim
    u = gradient(3, N, K, seed=6)
    u[1] = 0.0
    out = optim.orthogonalize(u, eps=eps)
    assert float(out[1].abs().max()) == 0.0
    assert bool(torch.isfinite(out).all())
    w = torch.randn((3, N, K), device="cuda")
    w1 = w[1].clone()
    optim.muon_update(w, u, torch.zeros_like(w), lr=0.5, scale=1.0, eps=eps)
    assert torch.equal(w[1], w1) and bool(torch.isfinite(w).all())
