"""Tensors that do not start at a 16-byte boundary (slices of a batch, of a
flat buffer) give the same bits as aligned copies of them, and outputs of that
kind are filled in place."""

import pytest
import torch

pytestmark = pytest.mark.gpu


def shifted(t, by=1):
    """t's values in a contiguous tensor that starts `by` elements behind a 16-byte boundary."""
    flat = torch.empty(t.numel() + by, dtype=t.dtype, device=t.device)
    out = flat[by:].view(t.shape)
    out.copy_(t)
    assert out.data_ptr() % 16 and out.is_contiguous()
    return out


@pytest.mark.parametrize("E", [10, 64])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_gate_of_a_slice_of_tokens(E, dtype):
    from mixture_experts_routed_route_gb300 import block
    g = torch.Generator("cuda").manual_seed(1)
    logits = torch.randn((70, E + 1), generator=g, device="cuda").to(dtype)
    bias = torch.randn(E + 1, generator=g, device="cuda")
    for view, b in ((logits[1:, :E], bias[:E]), (logits[:, 1:], bias[1:]), (logits[1:, 1:], None)):
        b0 = None if b is None else b.clone()
        ids, s = block.topk_gate(view.contiguous(), 3, renormalize=True, select_bias=b0)
        i1, s1 = block.topk_gate(view, 3, renormalize=True, select_bias=b)
        assert torch.equal(ids, i1) and torch.equal(s, s1)
        out_i, out_s = shifted(torch.zeros_like(ids)), shifted(torch.zeros_like(s))
        i2, s2 = block.topk_gate(view, 3, renormalize=True, select_bias=b, ids=out_i, scores=out_s)
        assert i2 is out_i and s2 is out_s and torch.equal(ids, i2) and torch.equal(s, s2)
        d = block.topk_gate_backward(view.contiguous(), ids, s, renormalize=True)
        assert torch.equal(d, block.topk_gate_backward(view, ids, s, renormalize=True))
        dl = shifted(torch.zeros_like(d))
        d1 = block.topk_gate_backward(view, shifted(ids), shifted(s), renormalize=True, d_logits=dl)
        assert d1 is dl and torch.equal(d, d1)


@pytest.mark.parametrize("D", [1411, 7, 2048])
@pytest.mark.parametrize("res", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("mode", ["channel", "group", "token"])
def test_norm_of_slices(D, res, mode):
    from mixture_experts_routed_route_gb300 import block
    T = 36
    g = torch.Generator("cuda").manual_seed(D)
    r = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    gate = r(*{"channel": (D,), "group": (4, D), "token": (T, 1)}[mode])
    whole = {"x": r(T, D).to(res), "b": r(T, D).bfloat16(), "dy": r(T, D).to(res), "dh": r(T, D).bfloat16(), "gate": gate,
             "wp": 1 + 0.1 * r(D), "wh": 1 + 0.1 * r(D)}
    part = {n: shifted(t) for n, t in whole.items()}

    def call(v, stats, y=None, h=None):
        kw = dict(gate=v["gate"], post_weight=v["wp"], pre_weight=v["wh"], residual_scale=0.9)
        return block.block_norm(v["x"], v["b"], stats=stats, y=y, h=h, **kw), block.block_norm_backward(
            v["x"] if y is not v["x"] else whole["x"], v["b"] if h is not v["b"] else whole["b"], stats, v["dy"], v["dh"], **kw)

    st0, st1 = torch.empty((2, T), device="cuda"), shifted(torch.zeros((2, T), device="cuda"))
    (y0, h0), g0 = call(whole, st0)
    (y1, h1), g1 = call(part, st1)
    assert torch.equal(y0, y1) and torch.equal(h0, h1) and torch.equal(st0, st1)
    assert all(torch.equal(p, q) for p, q in zip(g0, g1))
    (y2, h2), g2 = call(part, st1, y=part["x"], h=part["b"])     # in place
    assert y2 is part["x"] and h2 is part["b"] and torch.equal(y0, y2) and torch.equal(h0, h2)
    assert all(torch.equal(p, q) for p, q in zip(g0, g2))
    wide = torch.empty((T, D + 9), dtype=res, device="cuda")
    view = wide[:, 1:D + 1]
    view.copy_(whole["x"])
    y3, h3 = block.block_norm(view, whole["b"], gate=whole["gate"], post_weight=whole["wp"], pre_weight=whole["wh"], residual_scale=0.9)
    assert torch.equal(y0, y3) and torch.equal(h0, h3)
    # a norm alone, with and without an output for y
    y4, h4 = block.block_norm(part["dy"], pre_weight=part["wh"])
    assert y4 is part["dy"] and torch.equal(h4, block.block_norm(whole["dy"], pre_weight=whole["wh"])[1])
    y5, _ = block.block_norm(part["dy"], pre_weight=part["wh"], y=shifted(torch.zeros_like(whole["dy"])))
    assert torch.equal(y5, whole["dy"])


def test_norm_of_slices_on_a_side_stream():
    from mixture_experts_routed_route_gb300 import block
    x = torch.randn(3000, 1411, device="cuda")
    w = torch.ones(1411, device="cuda")
    want = block.block_norm(x[1:].clone(), pre_weight=w)[1]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = block.block_norm(x[1:], pre_weight=w, stream=side)[1]
    side.synchronize()
    assert torch.equal(got, want)


@pytest.mark.parametrize("N,K", [(33, 63), (300, 281), (64, 96)])
def test_updates_of_a_flat_buffer(N, K):
    from mixture_experts_routed_route_gb300 import optim
    from test_gpu_muon import gradient
    g = gradient(3, N, K)
    out = optim.orthogonalize(g)
    assert torch.equal(optim.orthogonalize(shifted(g)), out)
    o = shifted(torch.zeros_like(out))
    assert optim.orthogonalize(shifted(g), out=o) is o and torch.equal(o, out)
    w, m, c = torch.randn((3, N, K), device="cuda"), gradient(3, N, K, seed=2), torch.empty_like(out)
    w1, m1, c1 = shifted(w), shifted(m), shifted(c)
    optim.muon_update(w, g, m, lr=0.1, weight_bf16=c)
    optim.muon_update(w1, shifted(g), m1, lr=0.1, weight_bf16=c1)
    assert torch.equal(w, w1) and torch.equal(m, m1) and torch.equal(c, c1)
    with pytest.raises(ValueError, match="256"):
        optim.orthogonalize(g, workspace=optim.workspace(3, N, K)[16:])
