"""How precise the orthogonalised updates are before their own rounding, in
every run of matrices of a batch, and past 32-bit offsets.

X before its rounding is what a step on a zero FP32 weight leaves (lr = scale =
1, no decay, mu = 0: the weight becomes -X, exactly).  Its distance from 64
bits is compared with that of an emulation which rounds where the kernels do
and is exact elsewhere: operands to FP16 (X's hi half times 2^12, A and B times
2^9), X kept as hi + lo, the diagonal of B unrounded, and for smaller sizes up
to 256 the lo half in the apply product.  The kernels' FP32 sums flip some of
these roundings, so the two errors are different samples of the same sum of at
least 64 directions' independent roundings: their norms agree to a factor of 1
+ 2 / sqrt(64).  An operand less (B's diagonal rounded with the rest, or no lo
half) would be 1.4 to 2.3 times off on one of the two kinds of input below.
"""

import pytest
import torch

from test_gpu_muon import ABC, gradient, ns64

pytestmark = pytest.mark.gpu

FACTOR = 1.25


def emulate(u, eps=1e-7, diagonal=True, low=True):
    """The kernels' arithmetic on matrices [E, N, K] with sums in 64 bits;
    without B's FP32 diagonal or without the lo half: other designs."""
    if u.shape[1] > u.shape[2]:
        return emulate(u.transpose(1, 2), eps, diagonal, low).transpose(1, 2)
    half = lambda t, scale: (t * scale).half().double() / scale  # noqa: E731
    x = u.double()
    x = x / (x.square().sum((1, 2), keepdim=True).sqrt() + eps)
    a, b, c = ABC
    for _ in range(5):
        hi = half(x, 4096.0)
        lo = half(x - hi, 4096.0)
        A = half(hi @ hi.transpose(1, 2), 512.0)
        B = b * A + c * (A @ A)
        d = B.diagonal(dim1=1, dim2=2) * float(diagonal)
        B = half(B - torch.diag_embed(d), 512.0)
        x = (a + d)[:, :, None] * (hi + lo) + B @ (hi + lo if low and u.shape[1] <= 256 else hi)
    return x


def unrounded(u, **kw):
    from mixture_experts_routed_route_gb300 import optim
    w = torch.zeros(u.shape, device="cuda")
    optim.muon_update(w, u, torch.zeros_like(w), lr=1.0, mu=0.0, nesterov=False, weight_decay=0.0, scale=1.0, **kw)
    return -w


def off(got, ref):
    return (got.double() - ref).flatten(1).norm(dim=1) / ref.flatten(1).norm(dim=1)


@pytest.mark.parametrize("E,N,K", [(4, 64, 130), (4, 130, 64), (4, 128, 128), (3, 129, 127), (3, 100, 257), (8, 512, 256),
                                   (2, 256, 1030), (2, 300, 1000), (2, 1000, 300), (1, 641, 640), (1, 1000, 1531), (1, 1408, 2048)])
@pytest.mark.parametrize("kind", ["low rank and noise", "gaussian"])
def test_error_before_the_result_is_rounded(E, N, K, kind):
    u = gradient(E, N, K, seed=N + K) if kind != "gaussian" else torch.randn(
        (E, N, K), device="cuda", generator=torch.Generator("cuda").manual_seed(N))
    exact = ns64(u)
    got, emulated = off(unrounded(u), exact), off(emulate(u), exact)
    # the mean over the matrices of a batch: what one matrix's few roundings of
    # large elements add is part of the spread
    assert float(got.mean()) <= FACTOR * float(emulated.mean())


def test_long_contraction():
    """The tall 7168 x 2048 of a W2 gradient: 7168 terms a sum."""
    u = gradient(1, 7168, 2048, seed=1).bfloat16()
    exact = ns64(u)
    assert float(off(unrounded(u), exact)) <= FACTOR * float(off(emulate(u), exact))


@pytest.mark.parametrize("E,N,K", [(7, 320, 200), (5, 300, 281), (9, 512, 320)])
@pytest.mark.parametrize("matrices", [1, 2])
def test_updates_in_runs_of_matrices(E, N, K, matrices):
    """Weight, BF16 copy and momentum of every run of matrices, equal bit by bit to one run."""
    from mixture_experts_routed_route_gb300 import optim
    for dtype in (torch.float32, torch.bfloat16):
        grad, state = gradient(E, N, K, seed=1).bfloat16(), []
        for n in (E, matrices):
            w = torch.randn((E, N, K), device="cuda", generator=torch.Generator("cuda").manual_seed(3)).to(dtype)
            m = gradient(E, N, K, seed=2)
            c = torch.zeros((E, N, K), device="cuda", dtype=torch.bfloat16) if dtype is torch.float32 else None
            ws = optim.workspace(E, N, K, matrices=n)
            ws.fill_(0xFF)
            w0 = w.clone()
            optim.muon_update(w, grad, m, lr=0.02, weight_decay=0.1, weight_bf16=c, workspace=ws)
            assert all(not torch.equal(w[e], w0[e]) for e in range(E))
            assert c is None or torch.equal(c, w.bfloat16())
            state.append((w, m))
        assert torch.equal(state[0][0], state[1][0]) and torch.equal(state[0][1], state[1][1])


def test_stack_past_32_bit_offsets():
    """More than 2^32 bytes (and 2^31 elements) of a stack in several runs of matrices: the last ones are right."""
    from mixture_experts_routed_route_gb300 import optim
    E, N, K = 260, 4096, 2048
    grad = torch.empty((E, N, K), dtype=torch.bfloat16, device="cuda")
    g = torch.Generator("cuda").manual_seed(9)
    for e in range(E):
        grad[e].normal_(generator=g)
    weight = torch.zeros((E, N, K), dtype=torch.bfloat16, device="cuda")
    momentum = torch.zeros((E, N, K), device="cuda")
    optim.muon_update(weight, grad, momentum, lr=1.0, mu=0.5, nesterov=False, scale=1.0)
    tail = [t[-2:].clone() for t in (weight, grad, momentum)]
    assert torch.equal(tail[2], tail[1].float())
    w, m = torch.zeros_like(tail[0]), torch.zeros_like(tail[2])
    optim.muon_update(w, tail[1], m, lr=1.0, mu=0.5, nesterov=False, scale=1.0)
    assert torch.equal(w, tail[0]) and float(w.abs().max()) > 0.0
    out = optim.orthogonalize(grad)
    assert torch.equal(out[-2:], optim.orthogonalize(tail[1])) and torch.equal(out[-2:], -w)
    assert optim.error_bits() == 0
