"""Orthogonalised updates on the GPU against the iteration in 64 bits.

Bounds, all in the norm of a matrix.  The result's own BF16 rounding is at
most 2^-8 an element, about 2^-9 in norm.  Each of five steps rounds the operands of its products to FP16, at
most 2^-12 of each; what that perturbs reaches the result with a gain of at
most 2 for X's part and 2 for the polynomial's (the slope of a s + b s^3 +
c s^5 over its values is at most that where singular values end up), and a
step hands on the last one's perturbation with a gain of order one: 5 x 4 x
2^-12 < 5e-3.  Together below 7e-3 for |b|, |c| as here.
"""

import math

import pytest
import torch

pytestmark = pytest.mark.gpu

ABC = (3.4445, -4.7750, 2.0315)
BOUND = 7e-3


def ns64(u, steps=5, coefficients=ABC, eps=1e-7):
    table = coefficients if hasattr(coefficients[0], "__len__") else [coefficients] * steps
    x = u.double()
    x = x / (x.square().sum((1, 2), keepdim=True).sqrt() + eps)
    for a, b, c in table:
        if x.shape[1] <= x.shape[2]:
            q = x @ x.transpose(1, 2)
            x = a * x + (b * q + c * q @ q) @ x
        else:
            q = x.transpose(1, 2) @ x
            x = a * x + x @ (b * q + c * q @ q)
    return x


def gradient(E, N, K, seed=0, rank=32, noise=0.02):
    """A few strong directions over a weak full-rank part."""
    g = torch.Generator("cuda").manual_seed(seed)
    r = min(rank, N, K)
    rnd = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    return 1e-3 * ((rnd(E, N, r) * torch.logspace(0, -2, r, device="cuda")) @ rnd(E, r, K) + noise * rnd(E, N, K))


def off(got, ref):
    return float(((got.double() - ref).flatten(1).norm(dim=1) / ref.flatten(1).norm(dim=1).clamp(min=1e-300)).max())


SHAPES = [(1, 1, 1), (2, 1, 7), (3, 7, 1), (2, 3, 200), (4, 48, 48), (3, 64, 130), (2, 128, 128), (2, 129, 127), (3, 255, 256),
          (2, 256, 257), (5, 257, 100), (8, 512, 256), (1, 300, 1000), (2, 1000, 300), (1, 641, 640), (3, 1000, 1531),
          (2, 1408, 2048)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("E,N,K", SHAPES)
def test_orthogonalize(E, N, K, dtype):
    from mixture_experts_routed_route_gb300 import optim
    g = gradient(E, N, K, seed=N + K).to(dtype)
    out = optim.orthogonalize(g)
    assert out.dtype == torch.bfloat16 and off(out, ns64(g)) <= BOUND
    gauss = torch.randn((E, N, K), device="cuda", generator=torch.Generator("cuda").manual_seed(1)).to(dtype)
    assert off(optim.orthogonalize(gauss), ns64(gauss)) <= BOUND
    assert optim.error_bits() == 0


def test_singular_values_come_near_one():
    """What the operator is for: five steps take every singular value above
    1e-2 of the norm into [0.6, 1.3] (the polynomial's own band is [0.68,
    1.13]; the products' rounding moves it by less than the bound above)."""
    from mixture_experts_routed_route_gb300 import optim
    g = gradient(2, 96, 160, noise=0.3)
    s0 = torch.linalg.svdvals(g.double() / g.double().flatten(1).norm(dim=1)[:, None, None])
    s = torch.linalg.svdvals(optim.orthogonalize(g).double())
    s = s[s0 > 1e-2]
    assert float(s.min()) > 0.6 and float(s.max()) < 1.3


def test_steps_and_coefficients():
    from mixture_experts_routed_route_gb300 import optim
    g = gradient(3, 200, 333, noise=0.5)
    for steps in (1, 2, 3, 8):
        assert off(optim.orthogonalize(g, steps=steps), ns64(g, steps)) <= BOUND * max(1.0, steps / 5)
    table = [(2.0, -1.5, 0.5), (1.875, -1.25, 0.375), (3.4445, -4.7750, 2.0315)]
    assert off(optim.orthogonalize(g, steps=3, coefficients=table), ns64(g, 3, table)) <= BOUND
    assert off(optim.orthogonalize(g, steps=2, coefficients=(1.0, 0.0, 0.0)), ns64(g, 2, (1.0, 0.0, 0.0))) <= 2.0 ** -9


def test_zero_tiny_and_broken_matrices_keep_to_themselves():
    """A zero matrix gives zeros, one with a NaN gives NaN, and neither
    touches its neighbours; a norm below eps scales by 1/eps."""
    from mixture_experts_routed_route_gb300 import optim
    g = gradient(5, 300, 280)
    clean = optim.orthogonalize(g)
    g[1] = 0.0
    g[3, 5, 7] = math.nan
    out = optim.orthogonalize(g)
    assert float(out[1].abs().max()) == 0.0
    assert bool(torch.isnan(out[3]).all())
    for e in (0, 2, 4):
        assert torch.equal(out[e], clean[e])
    tiny = 1e-12 * gradient(2, 64, 64)
    assert off(optim.orthogonalize(tiny, eps=1e-9), ns64(tiny, eps=1e-9)) <= BOUND


def test_runs_of_matrices_and_workspaces_do_not_change_bits():
    from mixture_experts_routed_route_gb300 import abi, optim
    g = gradient(7, 320, 200).bfloat16()
    whole = optim.orthogonalize(g)
    for n in (1, 2, 3, 7):
        ws = optim.workspace(7, 320, 200, matrices=n)
        ws.fill_(0xFF)        # NaN everywhere: nothing of it may be read
        assert torch.equal(optim.orthogonalize(g, workspace=ws), whole), n
    small = torch.empty(optim.workspace(7, 320, 200, matrices=1).numel() - 1, dtype=torch.uint8, device="cuda")
    with pytest.raises(abi.MoEError) as e:
        optim.orthogonalize(g, workspace=small)
    assert e.value.status == abi.MOE_ERR_CAPACITY


# (smaller size at most 256) one to four CTA pairs a matrix, several rounds of
# matrices, and batches between them that the tiled kernels take
@pytest.mark.parametrize("E,N,K", [(1, 60, 250), (1, 200, 700), (1, 1000, 130), (9, 256, 513), (20, 900, 100), (37, 33, 65),
                                   (40, 256, 1030), (80, 300, 64), (90, 96, 200), (160, 140, 136), (230, 20, 30)])
def test_small_matrices_and_batches(E, N, K):
    from mixture_experts_routed_route_gb300 import optim
    g = gradient(E, N, K, seed=E).bfloat16()
    out = optim.orthogonalize(g)
    assert off(out, ns64(g)) <= BOUND
    one = optim.workspace(E, N, K, matrices=1)
    assert torch.equal(optim.orthogonalize(g, workspace=one), out)
    assert torch.equal(optim.orthogonalize(g), out)
    # the update's own tile walk, in place
    w = torch.randn((E, N, K), device="cuda", generator=torch.Generator("cuda").manual_seed(2))
    ref = 0.75 * w.double() - 0.5 * out.double()
    mom = torch.zeros_like(w)
    optim.muon_update(w, g, mom, lr=0.5, mu=0.0, nesterov=False, weight_decay=0.5, scale=1.0)
    # W - 0.5 X with X before its BF16 rounding: 0.5 x 2^-8 |X|, and FP32's rounding of W
    assert bool(((w.double() - ref).abs() <= 2.0 ** -9 * out.double().abs() + 2.0 ** -22 * (w.double().abs() + 1)).all())
    assert optim.error_bits() == 0


def test_tall_and_wide_agree():
    """The transposed input gives the transposed result, to the bound of each."""
    from mixture_experts_routed_route_gb300 import optim
    g = gradient(2, 192, 448)
    a = optim.orthogonalize(g)
    b = optim.orthogonalize(g.transpose(1, 2).contiguous())
    assert off(b.transpose(1, 2), a.double()) <= 2 * BOUND


@pytest.mark.parametrize("N,K", [(96, 160), (161, 90), (512, 256), (333, 1001)])
@pytest.mark.parametrize("wdtype,gdtype,nesterov,copy", [(torch.float32, torch.bfloat16, True, True),
                                                       (torch.float32, torch.float32, False, False),
                                                       (torch.bfloat16, torch.bfloat16, True, False),
                                                       (torch.bfloat16, torch.float32, False, False)])
def test_muon_update(N, K, wdtype, gdtype, nesterov, copy):
    from mixture_experts_routed_route_gb300 import optim
    E, lr, mu, wd, scale = 3, 2e-3, 0.9, 0.1, 4.0
    grad = gradient(E, N, K, seed=5).to(gdtype)
    mom = gradient(E, N, K, seed=6)
    w = (torch.randn((E, N, K), device="cuda") * K ** -0.5).to(wdtype)
    w16 = torch.empty((E, N, K), dtype=torch.bfloat16, device="cuda") if copy else None
    m64 = mu * mom.double() + grad.double()
    u = grad.double() + mu * m64 if nesterov else m64
    o = ns64(u)
    w64 = (1 - lr * wd) * w.double() - lr * scale * o
    m0 = mom.clone()
    optim.muon_update(w, grad, mom, lr=lr, mu=mu, nesterov=nesterov, weight_decay=wd, scale=scale, weight_bf16=w16)
    e = 2.0 ** -24
    assert bool(((mom.double() - m64).abs() <= 2 * e * (mu * m0.double().abs() + grad.double().abs())).all())
    upd = lr * scale * o
    for e_ in range(E):
        own = (2.0 ** -9 if wdtype == torch.bfloat16 else 3 * e) * w64[e_].norm()
        assert (w[e_].double() - w64[e_]).norm() <= own + 5e-3 * upd[e_].norm()
    if copy:
        assert torch.equal(w16, w.bfloat16())
    assert optim.error_bits() == 0


def test_streams_graphs_and_repeats():
    from mixture_experts_routed_route_gb300 import optim
    g = gradient(4, 300, 520).bfloat16()
    want = optim.orthogonalize(g)
    assert torch.equal(optim.orthogonalize(g), want)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = optim.orthogonalize(g, stream=side)
    torch.cuda.synchronize()
    assert torch.equal(got, want)
    ws = optim.workspace(4, 300, 520)
    out = torch.empty_like(want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        optim.orthogonalize(g, out=out, workspace=ws)
    for _ in range(2):
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)


def test_optimiser_object():
    """Muon keeps its state: two steps are two updates, with master weights or without."""
    from mixture_experts_routed_route_gb300 import optim
    shapes = [(2, 96, 128), (3, 130, 64)]
    for master in (False, True):
        ws = [torch.randn(s, device="cuda").bfloat16() for s in shapes]
        mine = [w.float() if master else w.clone() for w in ws]
        moms = [torch.zeros(s, device="cuda") for s in shapes]
        opt = optim.Muon(ws, lr=0.01, weight_decay=0.1, master=master)
        for k in range(2):
            grads = [gradient(*s, seed=k) for s in shapes]
            opt.step(grads)
            for w, g, m in zip(mine, grads, moms):
                optim.muon_update(w, g, m, lr=0.01, weight_decay=0.1)
        assert all(torch.equal(w, m.bfloat16()) for w, m in zip(ws, mine))


def test_empty_batch_and_refusals():
    from mixture_experts_routed_route_gb300 import abi, optim
    assert optim.orthogonalize(torch.empty(0, 4, 4, device="cuda")).shape == (0, 4, 4)
    x = torch.zeros(2, 8, 8, device="cuda")
    m = torch.zeros_like(x)
    for f in (lambda: optim.orthogonalize(x[0]), lambda: optim.orthogonalize(x.half()), lambda: optim.orthogonalize(x.transpose(1, 2)),
              lambda: optim.orthogonalize(x, steps=0), lambda: optim.orthogonalize(x, steps=17),
              lambda: optim.orthogonalize(x, coefficients=(1.0, 2.0)), lambda: optim.orthogonalize(x, out=torch.empty_like(x)),
              lambda: optim.orthogonalize(x, workspace=torch.zeros(4, device="cuda")),
              lambda: optim.muon_update(x, x[:1], m, lr=0.1), lambda: optim.muon_update(x, x.clone(), m.bfloat16(), lr=0.1),
              lambda: optim.muon_update(x.bfloat16(), x, m, lr=0.1, weight_bf16=x.bfloat16()),
              lambda: optim.muon_update(x, x.clone(), m, lr=0.1, weight_bf16=x.clone())):
        with pytest.raises(ValueError):
            f()
    for kw in (dict(eps=0.0), dict(coefficients=(99.0, 0.0, 0.0)), dict(eps=math.nan)):
        with pytest.raises(abi.MoEError) as e:
            optim.orthogonalize(x, workspace=optim.workspace(2, 8, 8), **kw)
        assert e.value.status == abi.MOE_ERR_INVALID_ARG
