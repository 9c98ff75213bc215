"""A refused call on the GPU, followed by a good one of the same shape."""

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("scale", [float("nan"), float("inf")])
def test_layer_norm_backward_after_a_refused_one(scale):
    from mixture_experts_routed_route_gb300 import abi, block
    T, D = (37, 520) if scale != scale else (41, 520)     # shapes of this test's own
    g = torch.Generator(device="cuda").manual_seed(1)
    y = torch.randn((T, D), generator=g, device="cuda")
    dh = torch.randn((T, D), generator=g, device="cuda").bfloat16()
    w = torch.ones(D, device="cuda")
    stats = torch.stack((y.mean(1), (y.var(1, correction=0) + 1e-5) ** -0.5))
    for kw in (dict(residual_scale=scale), dict(branch_scale=scale)):
        with pytest.raises(abi.MoEError) as e:
            block.layer_norm_backward(y, stats, dh, y, weight=w, bias=w, **kw)
        assert e.value.status == abi.MOE_ERR_INVALID_ARG
    got = block.layer_norm_backward(y, stats, dh, y, weight=w, bias=w)
    # column sums of T values in FP32: a rounding an addition, 2^-24 of the magnitudes each
    d = dh.double()
    assert bool(((got.dbias.double() - d.sum(0)).abs() <= T * 2.0 ** -24 * d.abs().sum(0)).all())
