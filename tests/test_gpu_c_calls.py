"""The calls around the layer through the C ABI's own binding (abi.py), as a
program without the torch wrappers makes them: the same bits as block.py's."""

import pytest
import torch

pytestmark = pytest.mark.gpu


def test_block_norm():
    from mixture_experts_routed_route_gb300 import abi, block
    T, D = 37, 520
    r = lambda *s: torch.randn(s, device="cuda")  # noqa: E731
    x, b, gate, wp, wh, dy, dh = r(T, D), r(T, D).bfloat16(), r(D), r(D).bfloat16(), r(D).bfloat16(), r(T, D), r(T, D).bfloat16()
    cfg = abi.moe_block_norm_config(T, D, abi.MOE_TYPE_FP32, abi.MOE_TYPE_BF16, abi.MOE_TYPE_FP32, abi.MOE_GATE_CHANNEL, 0,
                                    0.9, 1.1, 1e-6, 0.0, 0, 0, 0, 0)
    kw = dict(gate=gate, post_weight=wp, pre_weight=wh, residual_scale=0.9, branch_scale=1.1)
    st0, st1 = torch.zeros((2, T), device="cuda"), torch.zeros((2, T), device="cuda")
    y0, h0 = block.block_norm(x, b, stats=st0, **kw)
    y1, h1 = torch.empty_like(x), torch.empty_like(b)
    abi.moe_block_norm_forward(cfg, x, b, gate, wp, wh, y1, h1, st1)
    assert torch.equal(y0, y1) and torch.equal(h0, h1) and torch.equal(st0, st1)
    g0 = block.block_norm_backward(x, b, st0, dy, dh, **kw)
    g1 = [torch.empty_like(x), torch.empty_like(b), torch.empty_like(gate), torch.empty(D, device="cuda"), torch.empty(D, device="cuda")]
    ws = torch.empty(abi.moe_block_norm_workspace_bytes(cfg), dtype=torch.uint8, device="cuda")
    abi.moe_block_norm_backward(cfg, x, b, gate, wp, wh, st1, dy, dh, *g1, ws, ws.numel())
    assert all(torch.equal(p, q) for p, q in zip(g0, g1))
    with pytest.raises(abi.MoEError) as e:
        abi.moe_block_norm_backward(cfg, x, b, gate, wp, wh, st1, dy, dh, *g1, ws, ws.numel() - 1)
    assert e.value.status == abi.MOE_ERR_CAPACITY


def test_topk_gate():
    from mixture_experts_routed_route_gb300 import abi, block
    logits = torch.randn(50, 72, device="cuda")[:, :64]
    bias = torch.randn(64, device="cuda")
    cfg = abi.moe_topk_gate_config(50, 64, 5, abi.MOE_TYPE_FP32, abi.MOE_SCORE_SIGMOID, 1, 2.0, 72)
    kw = dict(score="sigmoid", renormalize=True, scale=2.0)
    i0, s0 = block.topk_gate(logits, 5, select_bias=bias, **kw)
    i1, s1, d1 = torch.empty_like(i0), torch.empty_like(s0), torch.empty((50, 64), device="cuda")
    abi.moe_topk_gate_forward(cfg, logits, bias, i1, s1)
    abi.moe_topk_gate_backward(cfg, logits, i1, s1, d1)
    assert torch.equal(i0, i1) and torch.equal(s0, s1)
    assert torch.equal(d1, block.topk_gate_backward(logits, i0, s0, **kw))
