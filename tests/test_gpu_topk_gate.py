"""The router's choice on the GPU: ids exactly as a stable sort of the FP32
keys gives them, scores and gradients against the formulas in 64 bits.

Bounds: a score is a quotient of exponentials (or a sigmoid) of differences up
to s = max |l - max l| that are rounded once: relative error below (64 + s) e,
e = 2^-24 (64: the exponential's and division's few units, a sum over 32 terms
a lane and a 5-level tree).  Gradients: the same relative to the sum of the
magnitudes that they add up, and u = 2^-8 (8 significant bits) of the result for BF16 logits.
"""

import math

import pytest
import torch

pytestmark = pytest.mark.gpu

E24 = 2.0 ** -24


def choose(logits, bias, K):
    key = logits.float() if bias is None else logits.float() + bias
    bad = ~((key < math.inf) & (logits.float() < math.inf)).all(1)
    top, ids = torch.sort(key, dim=1, descending=True, stable=True)
    on = (top[:, :K] > -math.inf) & ~bad[:, None]
    return torch.where(on, ids[:, :K], -1).to(torch.int32), on, bad


def values(logits, ids, on, score, renorm):
    """(scores before the scale, p over all experts or None, sigmoid slopes or None, what they were divided by)."""
    l = logits.double()
    g = torch.gather(l, 1, ids.clamp(min=0).long())
    if score == "sigmoid":
        v = torch.where(on, torch.sigmoid(g), 0.0)
        tot = v.sum(1, keepdim=True) + 1e-20
        return (v / tot if renorm else v), None, torch.where(on, torch.sigmoid(g) * torch.sigmoid(-g), 0.0), tot
    if renorm:
        m = torch.where(on, g, -math.inf).max(1, keepdim=True).values
        v = torch.where(on, torch.exp(g - m), 0.0)
        return v / v.sum(1, keepdim=True).clamp(min=1e-300), None, None, None
    m = l.max(1, keepdim=True).values
    p = torch.where(m > -math.inf, torch.exp(l - m), 0.0)
    p = p / p.sum(1, keepdim=True).clamp(min=1e-300)
    return torch.where(on, torch.gather(p, 1, ids.clamp(min=0).long()), 0.0), p, None, None


def spread(logits):
    l = logits.double()
    return float(torch.where(l > -math.inf, l.max(1, keepdim=True).values - l, 0.0).nan_to_num(0, 0, 0).max())


def make(T, E, kind, dtype, seed=0):
    g = torch.Generator("cuda").manual_seed(seed)
    l = 2.0 * torch.randn((T, E), generator=g, device="cuda")
    if kind == "ties":
        l = torch.randint(-2, 3, (T, E), generator=g, device="cuda").float()
    elif kind == "equal":
        l = torch.zeros((T, E), device="cuda")
        l[:, ::2] = -0.0
    elif kind == "masked":
        l = l.masked_fill(torch.rand((T, E), generator=g, device="cuda") < 0.8, -math.inf)
    elif kind == "lowest":
        l = l.masked_fill(torch.rand((T, E), generator=g, device="cuda") < 0.5, torch.finfo(dtype).min)
    if kind != "equal" and T > 2:
        l[1] = -math.inf      # a token whose every expert is masked
    return l.to(dtype)


CASES = [(1, 1, 1), (1, 384, 6), (5, 8, 2), (33, 31, 31), (64, 32, 32), (7, 33, 8), (130, 64, 6), (40, 100, 10),
         (50, 256, 8), (65, 384, 8), (20, 512, 32), (9, 1000, 4), (12, 1024, 32)]


@pytest.mark.parametrize("kind", ["plain", "ties", "equal", "masked", "lowest"])
@pytest.mark.parametrize("T,E,K", CASES)
def test_forward_and_backward(T, E, K, kind):
    from mixture_experts_routed_route_gb300 import block
    for i, dtype in enumerate((torch.float32, torch.bfloat16)):
        for score in ("softmax", "sigmoid"):
            for renorm in (False, True):
                logits = make(T, E, kind, dtype, seed=E + i)
                bias = None if (E + i + renorm) % 2 else torch.randn(E, device="cuda", generator=torch.Generator("cuda").manual_seed(E))
                ids, scores = block.topk_gate(logits, K, score=score, renormalize=renorm, scale=2.5, select_bias=bias)
                rid, on, _ = choose(logits, bias, K)
                assert torch.equal(ids, rid), (kind, dtype, score)
                v, p, slope, tot = values(logits, rid, on, score, renorm)
                rel = (64 + (spread(logits) if score == "softmax" and kind != "lowest" else 100.0)) * E24
                ref = 2.5 * v
                assert bool(((scores.double() - ref).abs() <= rel * ref + 1e-37).all()), (kind, dtype, score, renorm)
                # gradient of <scores, d>
                d = torch.randn((T, K), device="cuda", generator=torch.Generator("cuda").manual_seed(K))
                got = block.topk_gate_backward(logits, ids, d, score=score, renormalize=renorm, scale=2.5)
                dd = torch.where(on, 2.5 * d.double(), 0.0)
                if score == "sigmoid":
                    q = dd - (dd * v).sum(1, keepdim=True) if renorm else dd
                    mq = dd.abs() + (dd.abs() * v).sum(1, keepdim=True) if renorm else dd.abs()
                    dl, ml = (q / tot * slope, mq / tot * slope) if renorm else (q * slope, mq * slope)
                else:
                    dl, ml = v * dd, v * dd.abs()
                    if renorm:
                        dl, ml = dl - v * dl.sum(1, keepdim=True), ml + v * ml.sum(1, keepdim=True)
                out = torch.zeros((T, E), dtype=torch.float64, device="cuda")
                mag = torch.zeros_like(out)
                out.scatter_add_(1, rid.clamp(min=0).long(), torch.where(on, dl, 0.0))
                mag.scatter_add_(1, rid.clamp(min=0).long(), torch.where(on, ml, 0.0))
                if p is not None:
                    out, mag = out - p * dl.sum(1, keepdim=True), mag + p * ml.sum(1, keepdim=True)
                tol = (2.0 ** -8 if dtype == torch.bfloat16 else 0.0) * out.abs() + 2 * rel * mag + 1e-37
                assert bool(((got.double() - out).abs() <= tol).all()), (kind, dtype, score, renorm)


def test_gradient_against_differences():
    from mixture_experts_routed_route_gb300 import block
    T, E, K = 6, 40, 5
    logits = make(T, E, "plain", torch.float32, seed=4)
    logits[1] = torch.randn(E, device="cuda")
    d = torch.randn((T, K), device="cuda")
    v = torch.randn((T, E), device="cuda", dtype=torch.float64)
    for score in ("softmax", "sigmoid"):
        for renorm in (False, True):
            ids, _ = block.topk_gate(logits, K, score=score, renormalize=renorm)
            grad = block.topk_gate_backward(logits, ids, d, score=score, renormalize=renorm).double()
            f = lambda s: (values(logits.double() + s * v, ids, ids >= 0, score, renorm)[0] * d.double()).sum()  # noqa: E731
            slope = (f(1e-5) - f(-1e-5)) / 2e-5
            assert abs(float(slope - (grad * v).sum())) <= 1e-5 * float((grad * v).abs().sum()), (score, renorm)


def test_not_a_number_routes_nowhere():
    """NaN or +inf in a row: ids -1 and NaN scores and gradients there, other rows as before."""
    from mixture_experts_routed_route_gb300 import block
    logits = make(50, 64, "plain", torch.float32)
    ids0, s0 = block.topk_gate(logits, 4)
    logits[7, 3], logits[11, 60], logits[20, 5] = math.nan, math.inf, -math.nan
    ids, s = block.topk_gate(logits, 4)
    rows = [7, 11, 20]
    rest = [r for r in range(50) if r not in rows]
    assert bool((ids[rows] == -1).all()) and bool(torch.isnan(s[rows]).all())
    assert torch.equal(ids[rest], ids0[rest]) and torch.equal(s[rest], s0[rest])
    g = block.topk_gate_backward(logits, ids, torch.ones_like(s))
    assert bool(torch.isnan(g[rows]).all()) and bool(torch.isfinite(g[rest]).all())


def test_bad_and_repeated_ids_in_the_backward():
    """Ids outside [0, E) take no gradient; an id twice gets both terms."""
    from mixture_experts_routed_route_gb300 import block
    logits = make(4, 16, "plain", torch.float32)
    logits[1] = torch.randn(16, device="cuda")
    ids = torch.tensor([[3, 16], [5, 5], [-1, 2], [-7, 99]], dtype=torch.int32, device="cuda")
    d = torch.randn((4, 2), device="cuda")
    got = block.topk_gate_backward(logits, ids, d, score="sigmoid")
    s = torch.sigmoid(logits.double())
    ref = torch.zeros_like(s)
    ref[0, 3] = d[0, 0] * s[0, 3] * (1 - s[0, 3])
    ref[1, 5] = (d[1, 0] + d[1, 1]) * s[1, 5] * (1 - s[1, 5])
    ref[2, 2] = d[2, 1] * s[2, 2] * (1 - s[2, 2])
    assert torch.allclose(got.double(), ref, rtol=64 * E24, atol=64 * E24)


def test_strides_streams_and_graphs():
    from mixture_experts_routed_route_gb300 import block
    wide = make(70, 400, "plain", torch.float32)
    view = wide[:, :384]
    ids, s = block.topk_gate(view.contiguous(), 6, renormalize=True)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    i1, s1 = block.topk_gate(view, 6, renormalize=True, stream=side)
    g1 = block.topk_gate_backward(view, i1, s1, renormalize=True, stream=side)
    torch.cuda.synchronize()
    g0 = block.topk_gate_backward(view.contiguous(), ids, s, renormalize=True)
    assert torch.equal(ids, i1) and torch.equal(s, s1) and torch.equal(g0, g1)
    out_i, out_s = torch.empty_like(ids), torch.empty_like(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        block.topk_gate(view, 6, renormalize=True, ids=out_i, scores=out_s)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(ids, out_i) and torch.equal(s, out_s)
    e, es = block.topk_gate(view[:0], 6)
    assert e.shape == (0, 6) and es.shape == (0, 6)
    assert block.topk_gate_backward(view[:0].contiguous(), e, es).shape == (0, 384)


def test_rows_past_32_bit_offsets():
    from mixture_experts_routed_route_gb300 import block
    T, E = 2_200_000, 1024
    logits = torch.empty((T, E), dtype=torch.float32, device="cuda").normal_()
    ids, s = block.topk_gate(logits, 4)
    i1, s1 = block.topk_gate(logits[-5:].contiguous(), 4)
    assert torch.equal(ids[-5:], i1) and torch.equal(s[-5:], s1)
    g = block.topk_gate_backward(logits, ids, s)
    assert torch.equal(g[-5:], block.topk_gate_backward(logits[-5:].contiguous(), i1, s1))


def test_chosen_routes_run_through_the_layer():
    """The gate's output is what MoELayer.forward takes: a masked token's row is zero."""
    from mixture_experts_routed_route_gb300 import block
    from mixture_experts_routed_route_gb300.layer import MoELayer, PreparedWeight
    T, D, F, E, K = 64, 128, 128, 8, 2
    layer = MoELayer(T, D, F, E, K, "bf16", debug=True)
    w13 = PreparedWeight((torch.randn(E, 2 * F, D, device="cuda") * D ** -0.5).bfloat16(), "bf16")
    w2 = PreparedWeight((torch.randn(E, D, F, device="cuda") * F ** -0.5).bfloat16(), "bf16")
    logits = make(T, E, "plain", torch.float32)
    ids, scores = block.topk_gate(logits, K, renormalize=True)
    out = layer.forward(torch.randn(T, D, device="cuda").bfloat16(), ids, scores, w13, w2)
    assert float(out[1].abs().max()) == 0.0 and float(out[2].abs().max()) > 0.0
    assert layer.error_bits() == 0
    layer.close()


def test_wrapper_refusals():
    from mixture_experts_routed_route_gb300 import abi, block
    l = torch.zeros(4, 64, device="cuda")
    ids, s = block.topk_gate(l, 2)
    for f in (lambda: block.topk_gate(l.double(), 2), lambda: block.topk_gate(l[0], 2), lambda: block.topk_gate(l, 2, score="relu"),
              lambda: block.topk_gate(l.t(), 2), lambda: block.topk_gate(l, 2, select_bias=torch.zeros(63, device="cuda")),
              lambda: block.topk_gate(l, 2, select_bias=torch.zeros(64, device="cuda", dtype=torch.bfloat16)),
              lambda: block.topk_gate(l, 2, ids=ids.long()), lambda: block.topk_gate(l, 2, scores=s[:3]),
              lambda: block.topk_gate_backward(l, ids, s.double()), lambda: block.topk_gate_backward(l, ids[:3], s),
              lambda: block.topk_gate_backward(l, ids, s, d_logits=l.bfloat16())):
        with pytest.raises(ValueError):
            f()
    for k in (0, 33, 65):
        with pytest.raises(abi.MoEError) as e:
            block.topk_gate(l, k, ids=torch.empty((4, k), dtype=torch.int32, device="cuda"),
                            scores=torch.empty((4, k), device="cuda"))
        assert e.value.status == abi.MOE_ERR_INVALID_ARG
