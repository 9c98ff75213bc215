"""Dropout on the GPU against the mask's definition (tests/dropout_oracle.py).

The product with 1 / (1 - p) is one FP32 rounding of a factor that is itself
rounded once, an added residual one more; then the result's own rounding:
|got - ref| <= u |ref| + 3 2^-24 (|x| f + |residual|), u = 2^-8 for BF16, 0
for FP32 (counted)."""

import pytest
import torch

import dropout_oracle as oracle

pytestmark = pytest.mark.gpu

U = {torch.bfloat16: 2.0 ** -8, torch.float32: 0.0}


def reference(x, p, seed, step, site, residual=None):
    k, f = oracle.keep(*x.shape, p, seed, step, site)
    k = k.to(x.device)
    ref = torch.where(k, x.double() * f, 0.0)
    mag = torch.where(k, x.double().abs() * f, 0.0)
    if residual is not None:
        ref, mag = ref + residual.double(), mag + residual.double().abs()
    return ref, mag, k


def check(got, x, p, seed, step, site, residual=None):
    ref, mag, k = reference(x, p, seed, step, site, residual)
    tol = U[got.dtype] * ref.abs() + 3 * 2.0 ** -24 * mag
    assert bool(((got.double() - ref).abs() <= tol).all())
    if residual is None:
        assert bool((got[~k] == 0).all())


def make_rng(seed, step):
    return torch.tensor([seed, step], dtype=torch.int64, device="cuda")


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,D", [(1, 1), (1, 7), (3, 5), (128, 256), (17, 1411), (1, 8193), (1025, 64), (5, 8200)])
def test_dropout(T, D, dtype):
    from mixture_experts_routed_route_gb300 import block
    g = torch.Generator(device="cuda").manual_seed(T + D)
    for i, (p, seed, step, site) in enumerate([(0.1, 0x123456789ABCDEF, 17, 5), (0.5, -3, (1 << 35) + 1, 0),
                                               (0.9, 1 << 62, 2 ** 32 - 1, 2 ** 32 - 1)]):
        rng = make_rng(seed, step)
        x = torch.randn((T, D), generator=g, device="cuda").to(dtype)
        r = torch.randn((T, D), generator=g, device="cuda").to(dtype)
        check(block.dropout(x, p, rng, site=site), x, p, seed, step, site)
        check(block.dropout_backward(x, p, rng, site=site), x, p, seed, step, site)
        check(block.dropout(x, p, rng, site=site, residual=r), x, p, seed, step, site, r)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("D,pad", [(64, 8), (64, 3), (37, 3), (37, 8), (8, 8)])
def test_strided_rows(D, pad, dtype):
    """Rows of a wider tensor, results into one, whose other columns stay as they are."""
    from mixture_experts_routed_route_gb300 import block
    g = torch.Generator(device="cuda").manual_seed(D + pad)
    T = 33
    wide = [torch.randn((T, D + pad), generator=g, device="cuda").to(dtype) for _ in range(3)]
    x, r, out = (w[:, :D] for w in wide)
    before = wide[2].clone()
    got = block.dropout(x, 0.3, make_rng(5, 6), site=7, residual=r, out=out)
    assert got.data_ptr() == wide[2].data_ptr()
    check(got, x, 0.3, 5, 6, 7, r)
    assert torch.equal(wide[2][:, D:], before[:, D:])


def test_mask_does_not_depend_on_layout_or_type():
    from mixture_experts_routed_route_gb300 import block
    ones = torch.ones((19, 45), device="cuda")
    rng = make_rng(11, 12)
    a = block.dropout(ones, 0.4, rng, site=1) != 0
    wide = torch.ones((19, 50), device="cuda")
    b = block.dropout(wide[:, :45], 0.4, rng, site=1) != 0
    c = block.dropout(ones.bfloat16(), 0.4, rng, site=1) != 0
    d = block.dropout(ones.view(45, 19), 0.4, rng, site=1).view(19, 45) != 0    # the flat place counts
    assert torch.equal(a, b) and torch.equal(a, c) and torch.equal(a, d)


def test_dropped_places_hold_anything_and_ends_of_p():
    from mixture_experts_routed_route_gb300 import block
    rng = make_rng(1, 2)
    x = torch.randn((64, 72), device="cuda")
    k = oracle.keep(64, 72, 0.5, 1, 2, 0)[0].cuda()
    bad = torch.where(k, x, torch.tensor([float("nan"), float("inf")], device="cuda").repeat(64, 36))
    assert torch.equal(block.dropout(bad, 0.5, rng), block.dropout(x, 0.5, rng))
    assert bool((block.dropout(bad, 1.0, rng) == 0).all())
    assert torch.equal(block.dropout(x, 0.0, None), x)
    assert torch.equal(block.dropout(x, 1.0, rng, residual=x), x)
    assert block.dropout(x[:0], 0.5, rng).shape == (0, 72)


def test_in_place_and_unaligned():
    from mixture_experts_routed_route_gb300 import block
    rng = make_rng(3, 4)
    x = torch.randn((40, 56), device="cuda").bfloat16()
    want = block.dropout(x, 0.2, rng, residual=x)
    y = x.clone()
    assert block.dropout(y, 0.2, rng, residual=y, out=y) is y
    assert torch.equal(y, want)
    flat = torch.zeros(40 * 56 + 3, device="cuda", dtype=torch.bfloat16)
    view = flat[3:].view(40, 56)
    view.copy_(x)
    assert torch.equal(block.dropout(view, 0.2, rng, residual=view), want)
    out = block.dropout(view, 0.2, torch.tensor([0, 3, 4], device="cuda")[1:], residual=view, out=view)
    assert out is view and torch.equal(view, want) and bool((flat[:3] == 0).all())


def test_streams_and_graphs_draw_new_masks():
    """On another stream, and in a graph that advances the step itself."""
    from mixture_experts_routed_route_gb300 import block
    x = torch.ones((64, 256), device="cuda")
    rng = make_rng(9, 100)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    a = block.dropout(x, 0.5, rng, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    check(a, x, 0.5, 9, 100, 0)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        rng[1] += 1
        out = block.dropout(x, 0.5, rng)
    for step in (101, 102, 103):
        graph.replay()
        check(out, x, 0.5, 9, step, 0)


def test_elements_past_32_bits():
    """The last rows of a tensor with more than 2^32 elements take blocks past 2^29."""
    from mixture_experts_routed_route_gb300 import block
    D = 8192
    T = (1 << 32) // D + 3
    x = torch.ones((T, D), device="cuda", dtype=torch.bfloat16)
    block.dropout(x, 0.5, make_rng(21, 22), site=3, out=x)
    import numpy as np
    g = np.arange(T * D // 8 - 4 * D // 8, T * D // 8, dtype=np.uint64)
    w = oracle.philox((g & np.uint64(oracle.M32), g >> np.uint64(32), 3, 22), (21, 0))
    words = np.stack([np.broadcast_to(v, g.shape) for v in w], 1).astype("<u4").view("<u2").reshape(4, D)
    want = torch.from_numpy(words >= 32768).cuda()
    assert torch.equal(x[-4:] != 0, want)
