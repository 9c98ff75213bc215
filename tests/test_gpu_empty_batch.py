"""Calls on no tokens."""

import pytest
import torch

pytestmark = pytest.mark.gpu


def test_empty_batch_with_a_gate_of_every_element():
    from mixture_experts_routed_route_gb300 import block
    x = torch.empty((0, 64), device="cuda")
    b, w, gate = x.bfloat16(), torch.ones(64, device="cuda"), torch.empty((0, 64), device="cuda")
    st = torch.empty((2, 0), device="cuda")
    y, h = block.block_norm(x, b, gate=gate, post_weight=w, pre_weight=w, stats=st)
    assert y.shape == h.shape == (0, 64)
    r = block.block_norm_backward(x, b, st, x, b, gate=gate, post_weight=w, pre_weight=w)
    assert r.dgate.shape == (0, 64) and float(r.dpost_weight.abs().max()) == 0.0 == float(r.dpre_weight.abs().max())


def test_gate_rows_that_no_token_takes():
    """Without tokens a grouped gate's gradient is zero, whatever its number of rows; a gate without rows needs that."""
    from mixture_experts_routed_route_gb300 import block
    x = torch.empty((0, 64), device="cuda")
    b, gate = x.bfloat16(), torch.ones((3, 64), device="cuda")
    r = block.block_norm_backward(x, b, None, x, gate=gate)
    assert r.dgate.shape == (3, 64) and float(r.dgate.abs().max()) == 0.0
    with pytest.raises(ValueError):
        block.block_norm(torch.ones((4, 64), device="cuda"), torch.ones((4, 64), device="cuda").bfloat16(), gate=gate[:0])
