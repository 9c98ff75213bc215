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


@pytest.mark.parametrize("T", [2 ** 31, 2 ** 32 + 5])
def test_more_rows_than_the_library_counts_are_refused(T):
    from mixture_experts_routed_route_gb300 import block, optim
    x = torch.empty((T, 1), dtype=torch.bfloat16, device="cuda")
    with pytest.raises(ValueError, match="2.31"):
        block.topk_gate(x, 1)
    with pytest.raises(ValueError, match="2.31"):
        block.block_norm(x, pre_weight=torch.ones(1, device="cuda"))
    with pytest.raises(ValueError, match="2.31"):
        optim.orthogonalize(x.view(T, 1, 1))
