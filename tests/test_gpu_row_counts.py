"""Numbers of rows near and past 2^31."""

import pytest
import torch

pytestmark = pytest.mark.gpu


def test_gate_over_almost_two_to_the_31_rows():
    from mixture_experts_routed_route_gb300 import block
    T = 2 ** 31 - 3
    logits = torch.zeros((T, 1), dtype=torch.bfloat16, device="cuda")
    logits[-1] = 3.0
    ids, s = block.topk_gate(logits, 1, score="sigmoid")
    assert not bool(ids.any())
    assert bool((s[:-1] == 0.5).all()) and abs(float(s[-1, 0]) - 0.9525741) < 1e-6
