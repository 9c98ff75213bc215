"""The cross entropy over a vocabulary on the GPU against its definition in 64 bits.

Bounds, with u = 2^-8 (BF16's rounding) and e = 2^-23 (an FP32 addition that
may truncate, as a tensor core's accumulator).  A logit is a sum of D products
that are exact: its error is at most D e |scale| sum |h w| =: el.  lse: the
largest el of its row; exponentials are good to 2^-20 (the approximation's 2^-22
and the rounding of an argument below 64 that matters), sums to 256 serial
roundings: 2^-15 in all; and 4 roundings of values of its own size.  The
gradient g of a logit is relative to itself within el + 2^-15 + that of lse's
argument (64 2^-23), then rounded once: u.  dh and dweight: sums over V or T of
|g| |w|, each within g's relative error, plus as many accumulator steps e; their
own rounding u."""

import pytest
import torch

pytestmark = pytest.mark.gpu

U, E = 2.0 ** -8, 2.0 ** -23


class Case:
    def __init__(self, T, D, V, ignored=0, bad=0, wide=True, pad=0, scale=1.0, z=0.0, seed=0, spread=2.0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        r = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
        self.T, self.D, self.V, self.scale, self.z = T, D, V, scale, z
        self.weight = (spread * D ** -0.5 * r(V, D)).bfloat16()
        self.h = r(T, D + pad).bfloat16()[:, :D]
        self.targets = torch.randint(0, V, (T,), generator=g, device="cuda").to(torch.int64 if wide else torch.int32)
        order = torch.randperm(T, generator=g, device="cuda")
        self.targets[order[:ignored]] = -100
        self.targets[order[ignored:ignored + bad]] = V
        self.bad = self.targets == V
        self.on = (self.targets >= 0) & ~self.bad
        self.d_loss = (0.5 + torch.rand(T, generator=g, device="cuda")) / T
        self.kw = dict(logit_scale=scale, z_weight=z)

    def logits(self):
        h, w = self.h.double()[self.on], self.weight.double()
        return self.scale * h @ w.t(), self.D * E * self.scale * (h.abs() @ w.abs().t())

    def check_forward(self, loss, lse):
        assert bool((loss[~self.on & ~self.bad] == 0).all()) and bool((lse[~self.on] == 0).all())
        assert bool(loss[self.bad].isnan().all())
        if not bool(self.on.any()):
            return
        l, el = self.logits()
        t = self.targets[self.on].long()[:, None]
        ref = torch.logsumexp(l, 1)
        tol = el.max(1).values + 2.0 ** -15 + 4 * 2.0 ** -24 * ref.abs()
        assert bool(((lse[self.on].double() - ref).abs() <= tol).all())
        want = ref - l.gather(1, t)[:, 0] + self.z * ref ** 2
        tol = tol * (1 + 2 * self.z * ref.abs()) + el.gather(1, t)[:, 0] + 4 * 2.0 ** -24 * (want.abs() + self.z * ref ** 2)
        assert bool(((loss[self.on].double() - want).abs() <= tol).all())

    def lse32(self):
        out = torch.zeros(self.T, device="cuda")
        if bool(self.on.any()):
            out[self.on] = torch.logsumexp(self.logits()[0], 1).float()
        return out

    def check_backward(self, lse, dh, dweight):
        l, el = self.logits()
        t = self.targets[self.on].long()[:, None]
        ls, d = lse[self.on].double()[:, None], self.d_loss[self.on].double()[:, None] * self.scale
        p = torch.exp(l - ls) * (1 + 2 * self.z * ls)
        hot = torch.zeros_like(p).scatter_(1, t, 1.0)
        g = d * (p - hot)
        # the exponential's share of g carries its relative error, the whole of it the rounding's
        eg = d * p.abs() * (el + 2.0 ** -15 + 64 * E) * 1.1 + (U + 4 * 2.0 ** -24) * g.abs()
        h, w = self.h.double()[self.on], self.weight.double()
        if dh is not None:
            assert bool((dh[~self.on] == 0).all())
            ref, mag = g @ w, (eg + (self.V + 64) * E * g.abs()) @ w.abs()
            got = dh[self.on].double()
            assert bool(((got - ref).abs() <= mag + U * (ref.abs() + mag)).all()), float(((got - ref).abs() / (mag + U * ref.abs())).max())
        if dweight is not None:
            ref, mag = g.t() @ h, (eg + (self.T + 64) * E * g.abs()).t() @ h.abs()
            got = dweight.double()
            assert bool(((got - ref).abs() <= mag + U * (ref.abs() + mag)).all()), float(((got - ref).abs() / (mag + U * ref.abs())).max())


def error_bits():
    from mixture_experts_routed_route_gb300 import optim
    return optim.error_bits()


SHAPES = [(1, 8, 1), (1, 64, 300), (3, 8, 7), (5, 72, 1000), (130, 64, 513), (257, 136, 777), (300, 256, 2049),
          (64, 1408, 5003), (600, 512, 4096), (1000, 320, 10007), (513, 1032, 130)]


@pytest.mark.parametrize("T,D,V", SHAPES)
def test_forward(T, D, V):
    from mixture_experts_routed_route_gb300 import loss
    for i, (ign, bad, wide, pad, scale, z) in enumerate([(0, 0, True, 0, 1.0, 0.0), (T // 3, T // 7, False, 8, 0.5, 1e-3),
                                                        (T - 1, 0, True, 3, 2.0, 0.0)]):
        c = Case(T, D, V, ign, bad, wide, pad, scale, z, seed=i)
        c.check_forward(*loss.linear_cross_entropy(c.h, c.weight, c.targets, **c.kw))
    assert error_bits() == 0


@pytest.mark.parametrize("T,D,V", SHAPES)
def test_backward(T, D, V):
    from mixture_experts_routed_route_gb300 import loss
    for i, (ign, bad, wide, pad, scale, z) in enumerate([(0, 0, True, 0, 1.0, 0.0), (T // 3, T // 7, False, 8, 0.5, 1e-3),
                                                        (T - 1, 0, True, 3, 2.0, 0.0)]):
        c = Case(T, D, V, ign, bad, wide, pad, scale, z, seed=i)
        lse = c.lse32()
        for piece in (None, 1, 1024):
            ws = None if piece is None else loss.workspace(T, D, V, piece=piece)
            c.check_backward(lse, *loss.linear_cross_entropy_backward(c.h, c.weight, c.targets, lse, c.d_loss, workspace=ws,
                                                                      **c.kw))
    assert error_bits() == 0


@pytest.mark.parametrize("T,ignored", [(1, 0), (11, 0), (63, 0), (64, 0), (300, 236), (2000, 1995), (65, 0)])
def test_few_rows_lose_nothing_between_the_products(T, ignored):
    """Up to 64 rows that count: g is there to 2^-16, so a result is off by its own rounding and 2^-16 of the
    magnitudes beside what an FP32 g of these logits would be off by; one row more, and g is rounded to BF16."""
    from mixture_experts_routed_route_gb300 import loss
    c = Case(T, 256, 5000, ignored, seed=T)
    lse = c.lse32()
    dh, dw = loss.linear_cross_entropy_backward(c.h, c.weight, c.targets, lse, c.d_loss, **c.kw)
    c.check_backward(lse, dh, dw)
    if T - ignored > 64:
        return
    l, el = c.logits()
    ls, d = lse[c.on].double()[:, None], c.d_loss[c.on].double()[:, None]
    p = torch.exp(l - ls)
    g = d * (p - torch.zeros_like(p).scatter_(1, c.targets[c.on].long()[:, None], 1.0))
    eg = d * p * (el + 2.0 ** -15 + 64 * E) * 1.1 + (2.0 ** -16 + 8 * 2.0 ** -24) * g.abs()
    h, w = c.h.double()[c.on], c.weight.double()
    for got, ref, mag in ((dh[c.on], g @ w, (eg + (5000 + 64) * E * g.abs()) @ w.abs()),
                          (dw, g.t() @ h, (eg + (2 * T + 64) * E * g.abs()).t() @ h.abs())):
        assert bool(((got.double() - ref).abs() <= mag + U * (ref.abs() + mag)).all())


def test_one_gradient_alone():
    from mixture_experts_routed_route_gb300 import loss
    c = Case(200, 128, 3000, 20)
    lse = c.lse32()
    args = (c.h, c.weight, c.targets, lse, c.d_loss)
    dh, dw = loss.linear_cross_entropy_backward(*args, **c.kw)
    a, none = loss.linear_cross_entropy_backward(*args, need_dweight=False, **c.kw)
    assert none is None and torch.equal(a, dh)
    none, b = loss.linear_cross_entropy_backward(*args, need_dh=False, **c.kw)
    assert none is None and torch.equal(b, dw)
    oh, ow = torch.empty_like(dh), torch.empty_like(dw)
    got = loss.linear_cross_entropy_backward(*args, dh=oh, dweight=ow, **c.kw)
    assert got[0] is oh and got[1] is ow and torch.equal(oh, dh) and torch.equal(ow, dw)


def test_nothing_counts():
    from mixture_experts_routed_route_gb300 import loss
    c = Case(70, 64, 500, 60, 10)
    c.h.fill_(float("nan"))
    value, lse = loss.linear_cross_entropy(c.h, c.weight, c.targets)
    c.check_forward(value, lse)
    dh, dw = loss.linear_cross_entropy_backward(c.h, c.weight, c.targets, lse, c.d_loss)
    assert bool((dh == 0).all()) and bool((dw == 0).all())
    e = c.h[:0]
    value, lse = loss.linear_cross_entropy(e, c.weight, c.targets[:0])
    assert value.shape == lse.shape == (0,)
    dh, dw = loss.linear_cross_entropy_backward(e, c.weight, c.targets[:0], lse, value)
    assert dh.shape == (0, 64) and bool((dw == 0).all())
    assert error_bits() == 0


def test_ignored_rows_hold_anything():
    """NaN and infinities in ignored rows reach no result; those in a row that counts reach its own loss and gradient."""
    from mixture_experts_routed_route_gb300 import loss
    c = Case(300, 64, 1000, 100)
    want = loss.linear_cross_entropy(c.h, c.weight, c.targets)
    back = loss.linear_cross_entropy_backward(c.h, c.weight, c.targets, want[1], c.d_loss)
    h = c.h.clone()
    h[~c.on] = float("nan")
    h[~c.on, ::2] = float("inf")
    got = loss.linear_cross_entropy(h, c.weight, c.targets)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    got = loss.linear_cross_entropy_backward(h, c.weight, c.targets, want[1], c.d_loss)
    assert all(torch.equal(a, b) for a, b in zip(got, back))
    row = int(torch.nonzero(c.on)[5])
    h[row, 3] = float("nan")
    value, lse = loss.linear_cross_entropy(h, c.weight, c.targets)
    assert bool(value[row].isnan()) and int(value.isnan().sum()) == 1
    dh, _ = loss.linear_cross_entropy_backward(h, c.weight, c.targets, want[1], c.d_loss, need_dweight=False)
    assert bool(dh[row].isnan().all()) and int(dh.isnan().any(1).sum()) == 1


def test_large_logits():
    """Logits of several hundred: the maximum comes off before the exponentials."""
    from mixture_experts_routed_route_gb300 import loss
    c = Case(40, 64, 700, spread=120.0)
    value, lse = loss.linear_cross_entropy(c.h, c.weight, c.targets)
    assert float(lse.max()) > 300
    c.check_forward(value, lse)
    c.weight.mul_(0)
    value, lse = loss.linear_cross_entropy(c.h, c.weight, c.targets)
    assert float((value - torch.tensor(700.0).log()).abs().max()) < 1e-5


def test_gradients_against_differences():
    """Central differences of the loss in 64 bits along random directions."""
    from mixture_experts_routed_route_gb300 import loss
    c = Case(30, 48, 400, 5, z=1e-2, scale=0.7)
    lse = c.lse32()
    dh, dw = loss.linear_cross_entropy_backward(c.h, c.weight, c.targets, lse, c.d_loss, **c.kw)
    t = c.targets[c.on][:, None]

    def total(h, w):
        l = c.scale * h[c.on] @ w.t()
        ls = torch.logsumexp(l, 1)
        return float((c.d_loss[c.on].double() * (ls - l.gather(1, t)[:, 0] + c.z * ls ** 2)).sum())

    at = [c.h.double(), c.weight.double()]
    g = torch.Generator(device="cuda").manual_seed(3)
    for i, grad in enumerate((dh, dw)):
        v = torch.randn(at[i].shape, generator=g, device="cuda", dtype=torch.float64)
        hi, lo = list(at), list(at)
        hi[i], lo[i] = at[i] + 1e-4 * v, at[i] - 1e-4 * v
        want = (total(*hi) - total(*lo)) / 2e-4
        got = float((grad.double() * v).sum())
        # g's roundings and the results', each u relative at most, add up like independent ones: 6 deviations of both
        assert abs(got - want) <= 12 * U * float((grad.double() * v).norm()) + 1e-7, i


def test_streams_graphs_and_repeats():
    from mixture_experts_routed_route_gb300 import loss
    c = Case(300, 128, 3000, 40)
    want = loss.linear_cross_entropy(c.h, c.weight, c.targets)
    back = loss.linear_cross_entropy_backward(c.h, c.weight, c.targets, want[1], c.d_loss)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = loss.linear_cross_entropy(c.h, c.weight, c.targets, stream=side)
    again = loss.linear_cross_entropy_backward(c.h, c.weight, c.targets, got[1], c.d_loss, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, b) for a, b in zip(got + again, want + back))
    graph = torch.cuda.CUDAGraph()
    h, t = c.h.clone(), c.targets.clone()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        value, lse = loss.linear_cross_entropy(h, c.weight, t)
        dh, dw = loss.linear_cross_entropy_backward(h, c.weight, t, lse, c.d_loss)
    d = Case(300, 128, 3000, 250, seed=9)       # other tokens, another number that counts
    h.copy_(d.h)
    t.copy_(d.targets)
    graph.replay()
    want = loss.linear_cross_entropy(d.h, c.weight, d.targets)
    back = loss.linear_cross_entropy_backward(d.h, c.weight, d.targets, want[1], c.d_loss)
    assert all(torch.equal(a, b) for a, b in zip((value, lse, dh, dw), want + back))
    assert error_bits() == 0


def test_unaligned_tensors():
    from mixture_experts_routed_route_gb300 import loss
    c = Case(37, 64, 200, 4)
    want = loss.linear_cross_entropy(c.h, c.weight, c.targets)
    back = loss.linear_cross_entropy_backward(c.h, c.weight, c.targets, want[1], c.d_loss)

    def off(t):
        f = torch.zeros(t.numel() + 1, dtype=t.dtype, device="cuda")
        f[1:] = t.reshape(-1)
        return f[1:].view(t.shape)

    ol, os_, oh, ow = off(want[0] * 0), off(want[1] * 0), off(back[0] * 0), off(back[1] * 0)
    got = loss.linear_cross_entropy(off(c.h), off(c.weight), off(c.targets), loss=ol, lse=os_)
    assert got[0] is ol and torch.equal(ol, want[0]) and torch.equal(os_, want[1])
    got = loss.linear_cross_entropy_backward(off(c.h), off(c.weight), off(c.targets), os_, off(c.d_loss), dh=oh, dweight=ow)
    assert got[0] is oh and torch.equal(oh, back[0]) and torch.equal(ow, back[1])


def test_refusals():
    from mixture_experts_routed_route_gb300 import abi, loss
    c = Case(8, 64, 100)
    f, lse = loss.linear_cross_entropy, torch.zeros(8, device="cuda")
    for call in (lambda: f(c.h.float(), c.weight, c.targets), lambda: f(c.h, c.weight.float(), c.targets),
                 lambda: f(c.h, c.weight[:, :32], c.targets), lambda: f(c.h, c.weight.t(), c.targets),
                 lambda: f(c.h, c.weight, c.targets[:4]), lambda: f(c.h, c.weight, c.targets.float()),
                 lambda: f(c.h, c.weight, c.targets.cpu()), lambda: f(c.h, c.weight[:0], c.targets),
                 lambda: f(c.h, c.weight, c.targets, ignore_index=1 << 63), lambda: f(c.h, c.weight, c.targets, loss=lse[:4]),
                 lambda: loss.linear_cross_entropy_backward(c.h, c.weight, c.targets, lse.double(), lse),
                 lambda: loss.linear_cross_entropy_backward(c.h, c.weight, c.targets, lse, lse, need_dh=False,
                                                            need_dweight=False),
                 lambda: f(c.h, c.weight, c.targets, workspace=torch.zeros(1 << 20, device="cuda"))):
        with pytest.raises(ValueError):
            call()
    d = Case(8, 60, 100)
    with pytest.raises(abi.MoEError) as e:
        f(d.h, d.weight, d.targets)
    assert e.value.status == abi.MOE_ERR_UNSUPPORTED
    small = torch.empty(1024, dtype=torch.uint8, device="cuda")
    for call in (lambda: f(c.h, c.weight, c.targets, workspace=small),
                 lambda: loss.linear_cross_entropy_backward(c.h, c.weight, c.targets, lse, lse, workspace=small)):
        with pytest.raises(abi.MoEError) as e:
            call()
        assert e.value.status == abi.MOE_ERR_CAPACITY
    for kw in (dict(logit_scale=0.0), dict(z_weight=-1.0)):
        with pytest.raises(abi.MoEError) as e:
            f(c.h, c.weight, c.targets, **kw)
        assert e.value.status == abi.MOE_ERR_INVALID_ARG


def test_weights_past_32_bits():
    """A weight of more than 2^31 elements: the last entries' loss and gradient."""
    from mixture_experts_routed_route_gb300 import loss
    V, D, T = 303000, 7168, 4
    assert V * D > 1 << 31
    weight = torch.zeros((V, D), device="cuda", dtype=torch.bfloat16)
    g = torch.Generator(device="cuda").manual_seed(1)
    tail = 1000
    weight[-tail:] = (2 * D ** -0.5 * torch.randn((tail, D), generator=g, device="cuda")).bfloat16()
    h = torch.randn((T, D), generator=g, device="cuda").bfloat16()
    targets = torch.tensor([V - 1, V - 500, 0, V - 2], device="cuda")
    value, lse = loss.linear_cross_entropy(h, weight, targets)
    l = torch.zeros((T, V), device="cuda", dtype=torch.float64)
    l[:, -tail:] = h.double() @ weight[-tail:].double().t()
    ref = torch.logsumexp(l, 1)
    tol = D * E * float((h.double().abs() @ weight[-tail:].double().abs().t()).max()) + 2.0 ** -15
    assert float((lse - ref).abs().max()) <= tol
    assert float((value - (ref - l.gather(1, targets[:, None])[:, 0])).abs().max()) <= 2 * tol
    d = torch.full((T,), 0.25, device="cuda")
    dh, dw = loss.linear_cross_entropy_backward(h, weight, targets, lse, d)
    p = 0.25 * torch.exp(l[:, -tail:] - lse.double()[:, None])
    p[torch.arange(T, device="cuda"), (targets - (V - tail)).clamp(min=0)] -= 0.25 * (targets >= V - tail)
    want = p.t() @ h.double()
    mag = p.abs().t() @ h.double().abs()
    assert bool(((dw[-tail:].double() - want).abs() <= (3 * U + tol) * mag).all())
    assert bool((dw[1:-tail].float().abs() <= 1e-4).all())
    want, mag = p @ weight[-tail:].double(), p.abs() @ weight[-tail:].double().abs()
    assert bool(((dh.double() - want).abs() <= (3 * U + tol) * mag).all())
    assert error_bits() == 0
