"""Which schedules of coefficients the orthogonalised updates take (host
only): any of up to 16 in magnitude, and larger ones where every matrix stays
within the kernels' formats on the way."""

import pytest

from test_operators_cpu import muon_cfg

from mixture_experts_routed_route_gb300 import abi

STEEP = [(8.205, -22.902, 16.461), (4.066, -2.861, 0.518), (3.91, -2.823, 0.525), (3.286, -2.415, 0.485), (2.278, -1.62, 0.398)]
ABC = (3.4445, -4.7750, 2.0315)


def taken(table):
    c = muon_cfg(steps=len(table))
    for s, triple in enumerate(table):
        c.coefficients[s][:] = triple
    return abi.moe_muon_workspace_bytes(c, 1) > 0


def test_steep_schedules_that_stay_in_range():
    assert taken(STEEP)
    assert taken(STEEP + [STEEP[-1]] * 11)
    assert taken(STEEP[:1])
    assert taken([(10.5, 0.0, 0.0), (20.0, 0.0, 0.0)])               # A's 10.5^2
    assert taken([(0.5, 0.0, 0.0), (30.0, 0.0, 0.0)])                # 0.5, then the last step, whose result has no limit
    assert taken([(14.0, 0.0, 0.0), (0.0, -1.0, 0.0)]) and taken([(0.5, 0.0, 0.0), (20.0, -20.0, 10.0), (1.0, 0.0, 0.0)])


@pytest.mark.parametrize("table", [
    [(99.0, 0.0, 0.0), ABC],                                          # X
    [(11.3, 0.0, 0.0), (20.0, 0.0, 0.0)],                             # A's 11.3^2
    [(3.0, 0.0, 0.0), (20.0, 0.0, 4.0), ABC],                         # B's off-diagonal: 4 x 81 over 0
    [ABC, ABC, (3.4445, 17.0, 2.0315), ABC, ABC],
    [(8.29, -23.6, 17.3), (4.1, -2.95, 0.545), (3.95, -2.91, 0.552), (3.32, -2.49, 0.51), (2.3, -1.67, 0.419)],   # 0.5 % above 1 and it grows
    [(float("nan"), 0.0, 0.0)], [(17.0, float("inf"), 0.0)]])
def test_schedules_that_do_not(table):
    assert not taken(table)


def test_coefficients_up_to_16_are_up_to_the_caller():
    """They may grow the small singular values of a matrix that has no large one."""
    assert taken([(16.0, -16.0, 16.0)] * 16)
