"""Layer norm at a block boundary on the GPU against its formulas in 64 bits.

Bounds.  u = 2^-8 is BF16's unit of rounding (0 for FP32 results, whose own
rounding is a counted one), e = 2^-24 FP32's.  A result is one rounding of an
FP32 value that itself went through fewer than 128 roundings (at most 32 serial
additions a thread, a 10-level tree over threads and warps, some 40 products
and additions), each relative to the sum of the magnitudes of what it adds up:
|got - ref| <= u |ref| + 128 e mag, with mag from the same formulas on absolute
values.  A mean's error moves every element of its row, and an error of y - m
moves r, relative to itself, by as much as the row's errors relate to the row's
norm.  Sums over rows add a rounding a row (at most 700 of them, counted
apart)."""

import pytest
import torch

import dropout_oracle as oracle

pytestmark = pytest.mark.gpu

U = {torch.bfloat16: 2.0 ** -8, torch.float32: 0.0}
E24 = 2.0 ** -24
OPS = 128
ALPHA, BETA, EPS, SITE, SEED, STEP = 0.9, 1.2, 1e-5, 4, 77, 5


def near(name, got, ref, mag, ops=OPS):
    tol = U[got.dtype] * ref.abs() + ops * E24 * mag
    bad = (got.double() - ref).abs() > tol
    assert not bool(bad.any()), (name, int(bad.sum()), float(((got.double() - ref).abs() / tol.clamp(min=1e-300)).max()))


def avg(t):
    return t.mean(-1, keepdim=True)


class Case:
    def __init__(self, T, D, res, par, branch=True, p=0.0, affine=(True, True), pads=(0, 0, 0, 0, 0), seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        r = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
        rows = lambda t: t[:, :D]  # noqa: E731
        self.T, self.D, self.p = T, D, p
        self.x = rows((2.0 * r(T, D + pads[0]) + 0.7).to(res))
        self.branch = rows((0.5 * r(T, D + pads[1])).bfloat16()) if branch else None
        self.weight = (1 + 0.2 * r(D)).to(par) if affine[0] else None
        self.bias = (0.2 * r(D)).to(par) if affine[1] else None
        self.dy = rows(r(T, D + pads[2]).to(res))
        self.dh = rows(r(T, D + pads[3]).bfloat16())
        self.rng = torch.tensor([SEED, STEP], dtype=torch.int64, device="cuda")
        k, f = oracle.keep(T, D, p, SEED, STEP, SITE)
        self.keep = k.cuda().double() * f
        self.kw = dict(weight=self.weight, bias=self.bias, residual_scale=ALPHA, branch_scale=BETA, dropout=p,
                       rng=self.rng, site=SITE)

    def y64(self):
        y, m = ALPHA * self.x.double(), ALPHA * self.x.double().abs()
        if self.branch is not None:
            o = BETA * self.branch.double() * self.keep
            y, m = y + o, m + o.abs()
        return y, m

    def normed(self, y, my):
        """(n, magnitude of its errors, r, relative magnitude of r's errors)."""
        d, md = y - avg(y), my + avg(my)
        r = (avg(d * d) + EPS) ** -0.5
        rel = 1 + md.norm(dim=1, keepdim=True) / (d.norm(dim=1, keepdim=True) ** 2 + self.D * EPS).sqrt()
        return d * r, md * r + (d * r).abs() * rel, r, rel

    def affine64(self):
        w = 1.0 if self.weight is None else self.weight.double()
        b = torch.zeros(self.D, dtype=torch.float64, device="cuda") if self.bias is None else self.bias.double()
        return w, b

    def check_forward(self, y, h, stats):
        ry, my = self.y64()
        n, mn, r, rel = self.normed(ry, my)
        w, b = self.affine64()
        if y is not None:
            near("y", y, ry, my)
        near("h", h, n * w + b, mn * abs(w) + b.abs())
        if stats is not None:
            near("mean", stats[0], avg(ry)[:, 0], avg(my)[:, 0])
            near("r", stats[1], r[:, 0], (r * rel)[:, 0])

    def check_backward(self, y, grads, dy=True, branch=True):
        """At the y given, with its own statistics (those passed to the call are these, rounded)."""
        yd = y.double()
        n, mn, r, rel = self.normed(yd, yd.abs())
        w, _ = self.affine64()
        a, ma = self.dh.double() * w, self.dh.double().abs() * abs(w)
        s = r * (a - avg(a) - n * avg(a * n))
        ms = r * rel * (ma + avg(ma) + mn * avg(ma * n.abs()) + n.abs() * avg(ma * mn))
        if dy:
            s, ms = s + self.dy.double(), ms + self.dy.double().abs()
        near("dx", grads.dx, ALPHA * s, ALPHA * ms)
        if branch:
            near("dbranch", grads.dbranch, BETA * s * self.keep, BETA * ms * self.keep)
        else:
            assert grads.dbranch is None
        if self.weight is not None:
            near("dweight", grads.dweight, (self.dh.double() * n).sum(0), (self.dh.double().abs() * mn).sum(0), OPS + self.T)
        if self.bias is not None:
            near("dbias", grads.dbias, self.dh.double().sum(0), self.dh.double().abs().sum(0), OPS + self.T)


def stats_of(y):
    d = y.double()
    m = avg(d)
    return torch.stack((m[:, 0], (avg((d - m) ** 2) + EPS)[:, 0] ** -0.5)).float()


SHAPES = [(1, 1), (1, 7168), (3, 7), (5, 8), (17, 64), (33, 513), (6, 1000), (160, 2048), (301, 521), (2, 8192), (5, 8184),
          (3, 8191), (700, 24), (311, 1411), (161, 4095)]


@pytest.mark.parametrize("p", [0.0, 0.3])
@pytest.mark.parametrize("res", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,D", SHAPES)
def test_forward_and_backward(T, D, res, p):
    from mixture_experts_routed_route_gb300 import block
    for i, pads in enumerate([(0, 0, 0, 0), (8, 8, 16, 8), (3, 0, 1, 8)]):
        c = Case(T, D, res, torch.float32 if (T + i) % 2 else torch.bfloat16, p=p, pads=pads, seed=i)
        stats = torch.empty((2, T), device="cuda")
        y, h = block.layer_norm(c.x, c.branch, eps=EPS, stats=stats, **c.kw)
        assert y.is_contiguous() and h.is_contiguous()
        c.check_forward(y, h, stats)
        c.check_backward(y, block.layer_norm_backward(y, stats_of(y), c.dh, c.dy, **c.kw))


@pytest.mark.parametrize("p", [0.3, 1.0])
@pytest.mark.parametrize("res", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,D", [(7, 1024), (90, 4160), (305, 4104), (457, 5120), (609, 6152), (700, 7168), (500, 7176)])
def test_rows_of_one_group_a_cta(T, D, res, p):
    """Masks that go on from row to row, also between two calls whose generators differ."""
    from mixture_experts_routed_route_gb300 import block
    c = Case(T, D, res, torch.float32, p=p, pads=(0, 8, 0, 8, 0), seed=T)
    stats = torch.empty((2, T), device="cuda")
    y, h = block.layer_norm(c.x, c.branch, eps=EPS, stats=stats, **c.kw)
    c.check_forward(y, h, stats)
    st = stats_of(y)
    grads = block.layer_norm_backward(y, st, c.dh, c.dy, **c.kw)
    c.check_backward(y, grads)
    other = dict(c.kw, site=SITE + 1)
    block.layer_norm_backward(y, st, c.dh, c.dy, **other)
    again = block.layer_norm_backward(y, st, c.dh, c.dy, **c.kw)
    assert all(torch.equal(i, j) for i, j in zip(grads, again))


@pytest.mark.parametrize("T,D", [(9, 72), (9, 75), (200, 2048)])
def test_parts_left_out(T, D):
    """No branch, no weight, no bias, no dy, outputs of the caller's, rows of wider tensors."""
    from mixture_experts_routed_route_gb300 import block
    for affine in ((True, False), (False, True), (False, False)):
        c = Case(T, D, torch.float32, torch.float32, affine=affine)
        y, h = block.layer_norm(c.x, c.branch, eps=EPS, **c.kw)
        c.check_forward(y, h, None)
        c.check_backward(y, block.layer_norm_backward(y, stats_of(y), c.dh, None, **c.kw), dy=False)
    c = Case(T, D, torch.bfloat16, torch.bfloat16, branch=False)
    y, h = block.layer_norm(c.x, eps=EPS, **c.kw)
    c.check_forward(y, h, None)
    c.check_backward(y, block.layer_norm_backward(y, stats_of(y), c.dh, c.dy, branch=False, **c.kw), branch=False)
    plain, same = dict(c.kw, residual_scale=1.0), block.layer_norm(c.x, weight=c.weight)
    assert same[0] is c.x
    assert torch.equal(same[1], block.layer_norm(c.x, **dict(plain, bias=None), eps=1e-5)[1])
    for pad in (8, 5):
        c = Case(T, D, torch.float32, torch.bfloat16, p=0.25, pads=(pad, 3, 8, 5))
        wy = torch.full((T, D + pad), 7.0, device="cuda")
        wh = torch.full((T, D + pad), 7.0, device="cuda", dtype=torch.bfloat16)
        y, h = block.layer_norm(c.x, c.branch, eps=EPS, y=wy[:, :D], h=wh[:, :D], **c.kw)
        c.check_forward(y, h, None)
        assert bool((wy[:, D:] == 7).all()) and bool((wh[:, D:] == 7).all())
        c.check_backward(y, block.layer_norm_backward(y, stats_of(y), c.dh, c.dy, **c.kw))


def test_in_place_repeat_and_stream():
    from mixture_experts_routed_route_gb300 import block
    c = Case(333, 1000, torch.bfloat16, torch.bfloat16, p=0.1)
    y, h = block.layer_norm(c.x, c.branch, eps=EPS, **c.kw)
    x2, b2 = c.x.clone(), c.branch.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    block.layer_norm(x2, b2, eps=EPS, y=x2, h=b2, stream=side, **c.kw)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(x2, y) and torch.equal(b2, h)
    st = stats_of(y)
    a = block.layer_norm_backward(y, st, c.dh, c.dy, **c.kw)
    b = block.layer_norm_backward(y, st, c.dh, c.dy, **c.kw)
    assert all(torch.equal(i, j) for i, j in zip(a, b))


def test_same_mask_as_dropout():
    """The fused mask is dropout's on the contiguous branch, also where the branch is a slice."""
    from mixture_experts_routed_route_gb300 import block
    for D in (64, 77):
        rng = torch.tensor([3, 4], device="cuda")
        wide = torch.ones((21, D + 6), device="cuda", dtype=torch.bfloat16)
        x = torch.zeros((21, D), device="cuda")
        y, _ = block.layer_norm(x, wide[:, :D], dropout=0.5, rng=rng, site=9)
        d = block.dropout(torch.ones((21, D), device="cuda"), 0.5, rng, site=9)
        assert torch.equal(y, d)
        assert bool((block.layer_norm(x, wide[:, :D], dropout=1.0, rng=rng)[0] == 0).all())
        bad = torch.where(d == 0, float("nan"), 1.0).bfloat16()
        assert torch.equal(block.layer_norm(x, bad, dropout=0.5, rng=rng, site=9)[0], d)


def test_large_means_and_zero_rows():
    """The variance is taken about the mean: rows far from zero lose only what their own rounding loses."""
    from mixture_experts_routed_route_gb300 import block
    c = Case(8, 2048, torch.float32, torch.float32, branch=False)
    c.x = c.x * 1e-2 + 1000.0
    stats = torch.empty((2, 8), device="cuda")
    y, h = block.layer_norm(c.x, eps=EPS, stats=stats, **c.kw)
    c.check_forward(y, h, stats)
    y, h = block.layer_norm(torch.zeros((3, 40), device="cuda"), weight=torch.ones(40, device="cuda"),
                            bias=torch.arange(40.0, device="cuda"))
    assert torch.equal(h.float(), torch.arange(40.0, device="cuda").expand(3, 40))


def test_gradients_against_differences():
    """Directional differences of the formula in 64 bits against the kernel's gradients."""
    from mixture_experts_routed_route_gb300 import block
    c = Case(12, 96, torch.float32, torch.float32, p=0.4)
    y, _ = block.layer_norm(c.x, c.branch, eps=EPS, **c.kw)
    g = block.layer_norm_backward(y, stats_of(y), c.dh, c.dy, **c.kw)
    w, b = c.affine64()

    def loss(x, o, w, b):
        y = ALPHA * x + BETA * o * c.keep
        d = y - avg(y)
        h = d * (avg(d * d) + EPS) ** -0.5 * w + b
        return float((y * c.dy.double()).sum() + (h * c.dh.double()).sum())

    at = [c.x.double(), c.branch.double(), w, b]
    gen = torch.Generator(device="cuda").manual_seed(8)
    for i, grad in enumerate((g.dx, g.dbranch, g.dweight, g.dbias)):
        v = torch.randn(at[i].shape, generator=gen, device="cuda", dtype=torch.float64)
        hi, lo = list(at), list(at)
        hi[i], lo[i] = at[i] + 1e-4 * v, at[i] - 1e-4 * v
        want = (loss(*hi) - loss(*lo)) / 2e-4
        got = float((grad.double() * v).sum())
        # differences: O(1e-8); the BF16 gradient's rounding, as a sum of independent ones (six of their deviations)
        slack = 1e-6 * float((grad.double() * v).abs().sum()) + 6 * U[grad.dtype] * float((grad.double() * v).norm())
        assert abs(got - want) <= slack, i


def test_no_rows_and_unaligned():
    from mixture_experts_routed_route_gb300 import block
    w = torch.ones(40, device="cuda")
    x = torch.zeros((0, 40), device="cuda")
    y, h = block.layer_norm(x, x.bfloat16(), weight=w, bias=w)
    assert y.shape == h.shape == (0, 40)
    g = block.layer_norm_backward(y, torch.zeros((2, 0), device="cuda"), h, weight=w, bias=w)
    assert bool((g.dweight == 0).all()) and bool((g.dbias == 0).all()) and g.dx.shape == (0, 40)
    c = Case(19, 61, torch.float32, torch.float32, p=0.2)
    y, h = block.layer_norm(c.x, c.branch, eps=EPS, **c.kw)
    st = stats_of(y)
    want = block.layer_norm_backward(y, st, c.dh, c.dy, **c.kw)

    def off(t):
        f = torch.zeros(t.numel() + 1, dtype=t.dtype, device="cuda")
        f[1:] = t.reshape(-1)
        return f[1:].view(t.shape)

    kw = dict(c.kw, weight=off(c.weight), bias=off(c.bias), rng=off(c.rng))
    oy, oh, os_ = off(torch.zeros_like(y)), off(torch.zeros_like(h)), off(torch.zeros_like(st))
    y2, h2 = block.layer_norm(off(c.x), off(c.branch), eps=EPS, y=oy, h=oh, stats=os_, **kw)
    assert y2 is oy and torch.equal(oy, y) and torch.equal(oh, h)
    got = block.layer_norm_backward(off(y), off(st), off(c.dh), off(c.dy), **kw)
    assert all(torch.equal(i, j) for i, j in zip(got, want))


def test_captured_step_draws_new_masks():
    """Forward and backward in one graph that advances the step: each replay matches its own mask."""
    from mixture_experts_routed_route_gb300 import block
    c = Case(64, 256, torch.float32, torch.float32, p=0.5)
    ones = torch.ones((64, 256), device="cuda", dtype=torch.bfloat16)
    zero = torch.zeros((64, 256), device="cuda")
    block.layer_norm(zero, ones, **c.kw)
    stats = torch.empty((2, 64), device="cuda")
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        c.rng[1] += 1
        y, h = block.layer_norm(zero, ones, stats=stats, **c.kw)
        g = block.layer_norm_backward(y, stats, c.dh, c.dy, **c.kw)
    seen = []
    for step in (STEP + 1, STEP + 2):
        graph.replay()
        k = oracle.keep(64, 256, 0.5, SEED, step, SITE)[0].cuda()
        assert torch.equal(y != 0, k)
        assert bool((g.dbranch[~k] == 0).all())
        seen.append(k)
    assert not torch.equal(*seen)


def test_refusals():
    from mixture_experts_routed_route_gb300 import abi, block
    x = torch.zeros((4, 64), device="cuda")
    b, w, rng = x.bfloat16(), torch.ones(64, device="cuda"), torch.zeros(2, dtype=torch.int64, device="cuda")
    for call in (lambda: block.layer_norm(x, x), lambda: block.layer_norm(x, b, weight=w[:32]),
                 lambda: block.layer_norm(x, b, weight=w, bias=w.bfloat16()), lambda: block.layer_norm(x, dropout=0.5, rng=rng),
                 lambda: block.layer_norm(x, b, dropout=0.5), lambda: block.layer_norm(x, b, dropout=0.5, rng=rng.cpu()),
                 lambda: block.layer_norm(x.double()), lambda: block.layer_norm(x, b, stats=x),
                 lambda: block.layer_norm(x.t()), lambda: block.layer_norm(x, b, y=b), lambda: block.layer_norm(x, h=x),
                 lambda: block.layer_norm_backward(x, torch.zeros((2, 4), device="cuda"), x),
                 lambda: block.layer_norm_backward(x, torch.zeros((2, 5), device="cuda"), b),
                 lambda: block.layer_norm_backward(x, torch.zeros((2, 4), device="cuda"), b, branch=False, dropout=0.1, rng=rng),
                 lambda: block.dropout(x, 0.5, rng, residual=b), lambda: block.dropout(x, 0.5, rng, out=x[:2]),
                 lambda: block.dropout(x[0], 0.5, rng)):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(abi.MoEError):
        block.layer_norm(torch.zeros((2, 8193), device="cuda"))
