"""The norms around a block on the GPU against the formulas in 64 bits.

Bounds.  u = 2^-8 is BF16's unit of rounding (8 significant bits) (0 for FP32 results, whose own
rounding is one of the counted ones), e = 2^-24 FP32's.  A result is one
rounding of an FP32 value that itself went through fewer than 128 roundings
(at most 32 serial additions a thread, a 10-level tree over threads and warps,
and some 30 multiplications and additions), each relative to the sum of the
magnitudes of what it adds up: |got - ref| <= u |ref| + 128 e mag, with mag
from the same formulas on absolute values.  Sums over rows add one rounding a
row.  A 1/sqrt of a mean over D squares is relative to itself, as all its
terms are positive.
"""

import pytest
import torch

pytestmark = pytest.mark.gpu

U = {torch.bfloat16: 2.0 ** -8, torch.float32: 0.0}
E24 = 2.0 ** -24
OPS = 128


def rms(t, eps):
    return ((t * t).mean(-1, keepdim=True) + eps) ** -0.5


def rows_of(gate, T, mode):
    if gate is None:
        return 1.0
    if mode in ("channel", "token", "full"):
        return gate
    return gate.repeat_interleave(T // gate.shape[0], 0)


def forward64(x, b, g, wp, wh, mode, alpha, beta, eps, off):
    """(y, h, magnitude of y, magnitude of h) in 64 bits."""
    y, my = alpha * x, abs(alpha) * x.abs()
    if b is not None:
        p = b if wp is None else b * rms(b, eps) * (wp + off)
        p = beta * rows_of(g, x.shape[0], mode) * p
        y, my = y + p, my + p.abs()
    if wh is None:
        return y, None, my, None
    r = rms(y, eps)
    # an error of y moves r by as much, relative to the row's norm
    mh = (my + y.abs() * (my.norm(dim=1, keepdim=True) / y.norm(dim=1, keepdim=True).clamp(min=1e-300))) * r * (wh + off).abs()
    return y, y * r * (wh + off), my, mh


class Case:
    def __init__(self, T, D, res, par, mode, post, pre, pad=0, seed=0, groups=1):
        g = torch.Generator(device="cuda").manual_seed(seed)
        r = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
        self.mode, self.T, self.D = mode, T, D
        rows = lambda t: t[:, :D]  # noqa: E731
        self.x = rows((2.0 * r(T, D + pad)).to(res))
        self.b = None if mode == "nobranch" else rows((0.5 * r(T, D + pad)).bfloat16())
        shape = {"none": None, "nobranch": None, "channel": (D,), "group": (groups, D), "token": (T, 1), "full": (T, D)}[mode]
        self.g = None if shape is None else (0.7 + 0.3 * r(*shape)).to(par)
        self.wp = (1 + 0.2 * r(D)).to(par) if post else None
        self.wh = (1 + 0.2 * r(D)).to(par) if pre else None
        self.dy = rows(r(T, D + pad).to(res))
        self.dh = rows(r(T, D + pad).bfloat16()) if pre else None
        self.kw = dict(gate=self.g, post_weight=self.wp, pre_weight=self.wh, residual_scale=0.9, branch_scale=1.2,
                       weight_offset=0.25)
        self.eps = 1e-5

    def ref(self):
        d = lambda t: None if t is None else t.double()  # noqa: E731
        return forward64(d(self.x), d(self.b), d(self.g), d(self.wp), d(self.wh), self.mode, 0.9, 1.2, self.eps, 0.25)


def near(name, got, ref, mag, ops=OPS):
    """|got - ref| <= u |ref| + ops e mag, elementwise."""
    tol = U[got.dtype] * ref.abs() + ops * E24 * mag
    bad = (got.double() - ref).abs() > tol
    assert not bool(bad.any()), (name, int(bad.sum()), float(((got.double() - ref).abs() / tol.clamp(min=1e-300)).max()))


SHAPES = [(1, 1), (1, 7168), (3, 7), (5, 8), (17, 64), (33, 513), (6, 1000), (160, 2048), (301, 520), (2, 8192), (5, 8184),
          (3, 8191), (700, 24)]
GROUPS = {1: 1, 3: 3, 5: 5, 17: 17, 33: 11, 6: 2, 160: 4, 301: 7, 2: 1, 700: 7}


@pytest.mark.parametrize("mode", ["none", "channel", "group", "token", "full", "nobranch"])
@pytest.mark.parametrize("T,D", SHAPES)
def test_forward(T, D, mode):
    from mixture_experts_routed_route_gb300 import block
    for i, (post, pre) in enumerate([(1, 1), (0, 1), (1, 0), (0, 0)]):
        if mode == "nobranch" and (post or not pre):
            continue
        for res in (torch.bfloat16, torch.float32):
            c = Case(T, D, res, torch.float32 if (T + D + i) % 2 else torch.bfloat16, mode, post, pre, pad=(0, 8, 3)[i % 3],
                     seed=i, groups=GROUPS[T])
            stats = torch.zeros((2, T), device="cuda")
            y, h = block.block_norm(c.x, c.b, eps=c.eps, stats=stats, **c.kw)
            ry, rh, my, mh = c.ref()
            if mode != "nobranch":
                near("y", y, ry, my)
            if pre:
                near("h", h, rh, mh)
                near("r_y", stats[1], rms(ry, c.eps)[:, 0], rms(ry, c.eps)[:, 0] * (1 + my.norm(dim=1) / ry.norm(dim=1)))
            if post:
                near("r_o", stats[0], rms(c.b.double(), c.eps)[:, 0], rms(c.b.double(), c.eps)[:, 0])


def backward64(c):
    """The formulas' gradients in 64 bits, each with its magnitude."""
    alpha, beta, off, eps = 0.9, 1.2, 0.25, c.eps
    x, b = c.x.double(), None if c.b is None else c.b.double()
    T = c.T
    y, _, my, _ = c.ref()
    out = {}
    s, ms = c.dy.double(), c.dy.double().abs()
    if c.wh is not None:
        r = rms(y, eps)
        z, mz = y * r, my * r * (1 + my.norm(dim=1, keepdim=True) / y.norm(dim=1, keepdim=True).clamp(min=1e-300))
        a = c.dh.double() * (c.wh.double() + off)
        out["dpre_weight"] = ((c.dh.double() * z).sum(0), (c.dh.double().abs() * mz).sum(0))
        m = (a * z).mean(1, keepdim=True)
        s = s + r * (a - z * m)
        ms = ms + r * (a.abs() + mz * (a.abs() * mz).mean(1, keepdim=True)) * (1 + my.norm(dim=1, keepdim=True) / y.norm(dim=1, keepdim=True).clamp(min=1e-300))
    out["dx"] = (alpha * s, alpha * ms)
    if b is None:
        return out
    r_o = rms(b, eps) if c.wp is not None else torch.ones_like(b[:, :1])
    w = c.wp.double() + off if c.wp is not None else torch.ones(c.D, dtype=torch.float64, device="cuda")
    g = rows_of(None if c.g is None else c.g.double(), T, c.mode)
    n = b * r_o
    if c.g is not None:
        dg, mdg = beta * s * n * w, beta * ms * n.abs() * w.abs()
        if c.mode == "channel":
            dg, mdg = dg.sum(0), mdg.sum(0)
        elif c.mode == "token":
            dg, mdg = dg.sum(1, keepdim=True), mdg.sum(1, keepdim=True)
        elif c.mode == "group":
            dg, mdg = (t.view(c.g.shape[0], -1, c.D).sum(1) for t in (dg, mdg))
        out["dgate"] = (dg, mdg)
    bb, mb = beta * g * w * s, (beta * g * w).abs() * ms if c.g is not None else (beta * w).abs() * ms
    if c.wp is not None:
        out["dpost_weight"] = ((beta * g * s * n).sum(0), ((beta * g * n).abs() * ms).sum(0) if c.g is not None
                               else ((beta * n).abs() * ms).sum(0))
        m = (bb * n).mean(1, keepdim=True)
        out["dbranch"] = (r_o * (bb - n * m), r_o * (mb + n.abs() * (mb * n.abs()).mean(1, keepdim=True)))
    else:
        out["dbranch"] = (bb, mb)
    return out


@pytest.mark.parametrize("mode", ["none", "channel", "group", "token", "full", "nobranch"])
@pytest.mark.parametrize("T,D", SHAPES)
def test_backward(T, D, mode):
    from mixture_experts_routed_route_gb300 import block
    for i, (post, pre) in enumerate([(1, 1), (0, 1), (1, 0), (0, 0)]):
        if mode == "nobranch" and (post or not pre):
            continue
        for res in (torch.bfloat16, torch.float32):
            c = Case(T, D, res, torch.float32 if (T + D + i) % 2 else torch.bfloat16, mode, post, pre, pad=(0, 8, 3)[i % 3],
                     seed=10 + i, groups=GROUPS[T])
            stats = torch.zeros((2, T), device="cuda")
            block.block_norm(c.x, c.b, eps=c.eps, stats=stats, **c.kw)
            got = block.block_norm_backward(c.x, c.b, stats, c.dy, c.dh, **c.kw)
            for name, (ref, mag) in backward64(c).items():
                near((name, T, D, mode, post, pre, res), getattr(got, name), ref, mag, OPS + T)


def test_gradients_against_differences():
    """<gradient, direction> against a central difference of the 64-bit
    forward, for every input."""
    from mixture_experts_routed_route_gb300 import block
    for mode in ("channel", "group", "token", "full"):
        c = Case(12, 40, torch.float32, torch.float32, mode, 1, 1, seed=3, groups=4)
        stats = torch.zeros((2, 12), device="cuda")
        block.block_norm(c.x, c.b, eps=c.eps, stats=stats, **c.kw)
        got = block.block_norm_backward(c.x, c.b, stats, c.dy, c.dh, **c.kw)
        inputs = [c.x, c.b, c.g, c.wp, c.wh]
        for k, name in enumerate(("dx", "dbranch", "dgate", "dpost_weight", "dpre_weight")):
            v = torch.randn(inputs[k].shape, device="cuda", dtype=torch.float64, generator=torch.Generator("cuda").manual_seed(k))

            def loss(step):
                t = [q.double() for q in inputs]
                t[k] = t[k] + step * v
                y, h, _, _ = forward64(*t, mode, 0.9, 1.2, c.eps, 0.25)
                return (y * c.dy.double()).sum() + (h * c.dh.double()).sum()

            slope = (loss(1e-5) - loss(-1e-5)) / 2e-5
            grad = getattr(got, name).double()
            # BF16 gradients: u relative to each of the summed terms; the difference itself is good to 1e-8
            tol = U[getattr(got, name).dtype] * (grad * v).abs().sum() + 1e-5 * (grad * v).abs().sum()
            assert abs(float(slope - (grad * v).sum())) <= float(tol), (mode, name)


def test_no_pre_norm_gradient_and_final_norm():
    """dy missing (the norm before a head) and no dx wanted is the caller's; T = 0 gives zero gradients."""
    from mixture_experts_routed_route_gb300 import block
    c = Case(9, 96, torch.float32, torch.float32, "nobranch", 0, 1, seed=5)
    stats = torch.zeros((2, 9), device="cuda")
    block.block_norm(c.x, pre_weight=c.wh, residual_scale=0.9, weight_offset=0.25, eps=c.eps, stats=stats)
    got = block.block_norm_backward(c.x, None, stats, None, c.dh, pre_weight=c.wh, residual_scale=0.9, weight_offset=0.25)
    zero = block.block_norm_backward(c.x, None, stats, torch.zeros_like(c.x), c.dh, pre_weight=c.wh, residual_scale=0.9,
                                     weight_offset=0.25)
    assert torch.equal(got.dx, zero.dx) and torch.equal(got.dpre_weight, zero.dpre_weight)
    e = torch.empty((0, 96), device="cuda")
    eb = e.bfloat16()
    w = torch.ones(96, device="cuda")
    st = torch.empty((2, 0), device="cuda")
    y, h = block.block_norm(e, eb, gate=w, post_weight=w, pre_weight=w, stats=st)
    assert y.shape == (0, 96) and h.shape == (0, 96)
    r = block.block_norm_backward(e, eb, st, e, eb, gate=w, post_weight=w, pre_weight=w)
    assert all(float(t.abs().max()) == 0.0 for t in (r.dgate, r.dpost_weight, r.dpre_weight))


def test_zero_rows_and_infinities_stay_in_their_rows():
    from mixture_experts_routed_route_gb300 import block
    x = torch.randn(64, 256, device="cuda")
    b = torch.randn(64, 256, device="cuda").bfloat16()
    w = torch.ones(256, device="cuda")
    x[3], b[3] = 0.0, 0.0
    y0, h0 = block.block_norm(x, b, post_weight=w, pre_weight=w)
    assert float(h0[3].abs().max()) == 0.0 and float(y0[3].abs().max()) == 0.0
    x[5, 7], b[9, 1] = float("inf"), float("nan")
    y, h = block.block_norm(x, b, post_weight=w, pre_weight=w)
    keep = [r for r in range(64) if r not in (5, 9)]
    assert torch.equal(h[keep], h0[keep]) and torch.equal(y[keep], y0[keep])
    assert not bool(torch.isfinite(h[5].float()).all()) and bool(torch.isnan(h[9].float()).all())


def test_in_place_streams_graphs_and_repeats():
    """y over x and h over the branch; the same bits on a side stream, in a captured graph and again."""
    from mixture_experts_routed_route_gb300 import block
    for D in (2048, 1411):
        c = Case(257, D, torch.bfloat16, torch.bfloat16, "channel", 1, 1, seed=7)
        stats = torch.empty((2, 257), device="cuda")
        y, h = block.block_norm(c.x, c.b, eps=c.eps, stats=stats, **c.kw)
        g0 = block.block_norm_backward(c.x, c.b, stats, c.dy, c.dh, **c.kw)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        for s in (side, side.cuda_stream):
            st = torch.empty_like(stats)
            side.wait_stream(torch.cuda.current_stream())
            y1, h1 = block.block_norm(c.x, c.b, eps=c.eps, stats=st, stream=s, **c.kw)
            g1 = block.block_norm_backward(c.x, c.b, st, c.dy, c.dh, stream=s, **c.kw)
            torch.cuda.synchronize()
            assert torch.equal(y, y1) and torch.equal(h, h1) and torch.equal(stats, st)
            assert all(torch.equal(p, q) for p, q in zip(g0, g1))
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            y2, h2 = block.block_norm(c.x, c.b, eps=c.eps, **c.kw)
            g2 = block.block_norm_backward(c.x, c.b, stats, c.dy, c.dh, **c.kw)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, y2) and torch.equal(h, h2) and all(torch.equal(p, q) for p, q in zip(g0, g2))
        x, b = c.x.clone(), c.b.clone()
        y3, h3 = block.block_norm(x, b, eps=c.eps, y=x, h=b, **c.kw)
        assert y3 is x and h3 is b and torch.equal(x, y) and torch.equal(b, h)


def test_rows_past_32_bit_offsets():
    """More than 2^32 bytes of rows: the last ones are right."""
    from mixture_experts_routed_route_gb300 import block
    T, D = 270_000, 8192
    x = torch.empty((T, D), dtype=torch.bfloat16, device="cuda").normal_()
    b = torch.empty((T, D), dtype=torch.bfloat16, device="cuda").normal_()
    w = torch.ones(D, device="cuda")
    stats = torch.empty((2, T), device="cuda")
    y, h = block.block_norm(x, b, post_weight=w, pre_weight=w, stats=stats)
    y1, h1 = block.block_norm(x[-3:].contiguous(), b[-3:].contiguous(), post_weight=w, pre_weight=w)
    assert torch.equal(y[-3:], y1) and torch.equal(h[-3:], h1)
    r = block.block_norm_backward(x, b, stats, x, b, post_weight=w, pre_weight=w)
    r1 = block.block_norm_backward(x[-3:].contiguous(), b[-3:].contiguous(), stats[:, -3:].contiguous(),
                                   x[-3:].contiguous(), b[-3:].contiguous(), post_weight=w, pre_weight=w)
    assert torch.equal(r.dx[-3:], r1.dx) and torch.equal(r.dbranch[-3:], r1.dbranch)


def test_wrapper_refusals():
    from mixture_experts_routed_route_gb300 import block
    x = torch.zeros(4, 64, device="cuda")
    b = x.bfloat16()
    w = torch.ones(64, device="cuda")
    bad = [lambda: block.block_norm(x),                                            # nothing to compute
           lambda: block.block_norm(x.half(), pre_weight=w),
           lambda: block.block_norm(x[0], pre_weight=w),
           lambda: block.block_norm(x, x, post_weight=w),                          # an FP32 branch
           lambda: block.block_norm(x, b[:3], post_weight=w),
           lambda: block.block_norm(x, post_weight=w),
           lambda: block.block_norm(x, gate=w),
           lambda: block.block_norm(x, b, gate=torch.ones(3, 64, device="cuda")),  # 3 does not divide 4
           lambda: block.block_norm(x, b, gate=torch.ones(5, device="cuda")),
           lambda: block.block_norm(x, b, gate=w.double()),
           lambda: block.block_norm(x, pre_weight=w[:63]),
           lambda: block.block_norm(x, b, pre_weight=w, post_weight=w.bfloat16()),  # two weight types
           lambda: block.block_norm(x.t(), pre_weight=w),
           lambda: block.block_norm(x[:1].expand(4, 64), pre_weight=w),            # overlapping rows
           lambda: block.block_norm(x, b, h=b),                                    # no norm for h
           lambda: block.block_norm(x, pre_weight=w, stats=torch.zeros(4, 2, device="cuda")),
           lambda: block.block_norm(x, pre_weight=w, y=b),
           lambda: block.block_norm(x, pre_weight=w.cpu()),
           lambda: block.block_norm_backward(x, b, None, x, b, pre_weight=w),
           lambda: block.block_norm_backward(x, b, None, x, b),
           lambda: block.block_norm_backward(x, b, None, None)]
    for i, f in enumerate(bad):
        with pytest.raises(ValueError):
            f()
            raise AssertionError(i)
