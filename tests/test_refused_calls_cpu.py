"""A refused call leaves nothing behind that a later good call would meet (no GPU)."""

import pytest
import torch

from mixture_experts_routed_route_gb300 import abi, block, loss


class Sizes:
    """The library's size query: 0 for a configuration it refuses."""

    def moe_layer_norm_workspace_bytes(self, ref):
        cfg = ref._obj
        return 0 if cfg.residual_scale != cfg.residual_scale else 4096


def norm_cfg(scale):
    return abi.moe_layer_norm_config(123, 457, abi.MOE_TYPE_BF16, abi.MOE_TYPE_BF16, scale, 1.0, 1e-5, 0, 0.0, 0, 0, 0, 0)


def test_the_size_of_a_refused_layer_norm_is_not_remembered(monkeypatch):
    monkeypatch.setattr(block, "_LIB", Sizes())
    monkeypatch.setattr(block, "_norm_bytes", {})
    dev = torch.device("cpu")
    assert block._layer_norm_workspace(norm_cfg(float("nan")), dev).numel() == 0
    assert block._layer_norm_workspace(norm_cfg(1.0), dev).numel() == 4096
    assert block._layer_norm_workspace(norm_cfg(float("nan")), dev).numel() == 4096     # of the shape; the call refuses it
    assert len(block._norm_bytes) == 1


@pytest.mark.parametrize("sizes", [(1 << 32, 64, 100), ((1 << 32) + 4, 64, 100), (4, (1 << 32) + 64, 100),
                                   (4, 64, (1 << 32) + 100), (1 << 31, 64, 100), (-1, 64, 100), (4, 0, 100), (4, 64, 0)])
def test_a_cross_entropy_workspace_of_sizes_that_no_call_takes(sizes):
    """Sizes that 32 bits would cut off to others are refused, not answered for those."""
    with pytest.raises(ValueError, match="sizes"):
        loss.workspace(*sizes)
