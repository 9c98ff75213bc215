"""That the precision test of the orthogonalised updates can tell designs
apart: the emulation of a kernel that rounds B's diagonal with the rest, or
reads no lo half, fails its bound on one of its kinds of input (no GPU)."""

import pytest
import torch

from test_gpu_muon_precision import FACTOR, emulate, ns64, off


def inputs(E, N, K):
    g = torch.Generator().manual_seed(N + K)
    rnd = lambda *s: torch.randn(s, generator=g)  # noqa: E731
    r = min(32, N, K)
    return 1e-3 * ((rnd(E, N, r) * torch.logspace(0, -2, r)) @ rnd(E, r, K) + 0.02 * rnd(E, N, K)), rnd(E, N, K)


@pytest.mark.parametrize("E,N,K", [(4, 64, 130), (4, 128, 128), (3, 100, 257), (4, 256, 512), (1, 300, 1000)])
def test_other_designs_exceed_the_bound(E, N, K):
    low_rank, gauss = inputs(E, N, K)
    mean = lambda u, **kw: float(off(emulate(u, **kw), ns64(u)).mean())  # noqa: E731
    assert mean(gauss, diagonal=False) > FACTOR * mean(gauss)
    if min(N, K) <= 256:
        assert mean(low_rank, low=False) > FACTOR * mean(low_rank)
    assert mean(low_rank) < 1e-3 and mean(gauss) < 1.2e-3            # what the header says of the kernels
