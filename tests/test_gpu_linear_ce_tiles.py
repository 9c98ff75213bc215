"""Paths of the cross entropy that long batches, wide rows and odd vocabularies reach: rows found and packed by kernels
of their own (more than 1024 tokens), second groups of eight row tiles, sums in segments, narrow last tiles.  Bounds are
those of test_gpu_linear_ce.py, of test_gpu_linear_ce_precision.py for a logit's sums."""

import math

import pytest
import torch

from test_gpu_linear_ce import Case, error_bits
from test_gpu_linear_ce_precision import confident, truncated_logit

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T,D,V,ignored,bad", [(2600, 64, 1000, 0, 0), (2600, 72, 1100, 500, 41), (3100, 1032, 520, 700, 9),
                                               (1025, 40, 300, 1, 1), (2049, 64, 257, 2048 - 60, 0), (5000, 16, 129, 100, 30),
                                               (1500, 8, 5, 1400, 100)])
def test_many_row_tiles(T, D, V, ignored, bad):
    """Some ignored and some out of range, before and after token 1024."""
    from mixture_experts_routed_route_gb300 import loss
    for i, (wide, pad, scale, z) in enumerate([(True, 0, 1.0, 0.0), (False, 3, 0.5, 1e-3)]):
        c = Case(T, D, V, ignored, bad, wide, pad, scale, z, seed=i)
        if ignored:
            assert bool((~c.on[:1024]).any()) and bool((~c.on[1024:]).any() or T < 1100)
        c.check_forward(*loss.linear_cross_entropy(c.h, c.weight, c.targets, **c.kw))
        lse = c.lse32()
        for piece in (None, 256):
            ws = None if piece is None else loss.workspace(T, D, V, piece=piece)
            c.check_backward(lse, *loss.linear_cross_entropy_backward(c.h, c.weight, c.targets, lse, c.d_loss, workspace=ws,
                                                                      **c.kw))
    assert error_bits() == 0


@pytest.mark.parametrize("T", [1, 33, 65, 300, 1100])
@pytest.mark.parametrize("D", [1088, 2056, 4104])
@pytest.mark.parametrize("V", [1000, 1100, 130, 120])
def test_segments_and_last_tiles(T, D, V):
    """Two to five segments, the last a stage or less, and last tiles of 232, 76, 130 and 120 columns."""
    from mixture_experts_routed_route_gb300 import loss
    c = Case(T, D, V, T // 5, T // 50, pad=8, z=1e-3, seed=D + V)
    c.check_forward(*loss.linear_cross_entropy(c.h, c.weight, c.targets, **c.kw))
    lse = c.lse32()
    c.check_backward(lse, *loss.linear_cross_entropy_backward(c.h, c.weight, c.targets, lse, c.d_loss, **c.kw))
    assert error_bits() == 0


@pytest.mark.parametrize("T,steps", [(5, 16), (64, 16), (65, 64), (300, 64)])
@pytest.mark.parametrize("D,V", [(7168, 1000), (7168, 900), (4104, 1100), (2048, 700)])
def test_logits_are_summed_in_segments(T, steps, D, V):
    """lse is nearly the target's logit here: off by what cutting off loses in sums of 256 (up to 64 tokens) or 1024
    elements, one way only, beside lse's own roundings; one sum of 7168 would lose seven times as much."""
    from mixture_experts_routed_route_gb300 import loss
    h, weight, targets = confident(T, D, V, 40.0, 40.0 - 8.1 - math.log(V), T + D)
    logits = h.double() @ weight.double().t()
    ref = torch.logsumexp(logits, 1)
    _, lse = loss.linear_cross_entropy(h, weight, targets)
    off = ref - lse.double()
    # roundings of values up to 64 in base 2 and of 40: as the forward's own in test_gpu_linear_ce_precision.py
    own = 2.0 ** -19 * (1 + 2 * math.log(2)) + 2.0 ** -20
    most = truncated_logit(h.double(), weight.double()[targets], steps)
    print(T, D, "low by", float(off.mean() / 40), "at most", float((most + own).max() / 40))
    assert bool((off <= most + own).all()) and bool((off >= -own - D / 16 / steps * 2.0 ** -19).all())
    assert error_bits() == 0
