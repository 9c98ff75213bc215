"""The range of the orthogonalised updates: singular values up to the stated
limits on the way, on the tiled and the small kernel, wide and tall.

Bounds.  Where every product is exact in the kernel's formats (powers of two
and small whole numbers) the result has to be the exact value rounded to
BF16.  Else as in test_gpu_muon.py."""

import pytest
import torch

from test_gpu_muon import BOUND, ns64, off

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
