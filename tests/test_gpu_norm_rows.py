"""The norms around a block where every group of warps takes many rows: the
ring of rows in flight, sums over rows, and grouped gates with slabs of many
rows and with more gate rows than there are groups.  Formulas and bounds are
test_gpu_block_norm.py's."""

import pytest
import torch

from test_gpu_block_norm import OPS, Case, backward64, near, rms

pytestmark = pytest.mark.gpu

# at most 15 groups of warps share an SM: more rows than all of them take at once
SHAPES = [(4000, 1411), (3001, 2056), (2500, 7168), (4800, 1024), (9000, 24), (2503, 8191)]


def groups_at_most():
    return 15 * torch.cuda.get_device_properties(0).multi_processor_count


def check(c, T, D, mode):
    from mixture_experts_routed_route_gb300 import block
    stats = torch.zeros((2, T), device="cuda")
    y, h = block.block_norm(c.x, c.b, eps=c.eps, stats=stats, **c.kw)
    ry, rh, my, mh = c.ref()
    near(("y", mode), y, ry, my)
    near(("h", mode), h, rh, mh)
    near("r_y", stats[1], rms(ry, c.eps)[:, 0], rms(ry, c.eps)[:, 0] * (1 + my.norm(dim=1) / ry.norm(dim=1)))
    near("r_o", stats[0], rms(c.b.double(), c.eps)[:, 0], rms(c.b.double(), c.eps)[:, 0])
    del ry, rh, my, mh
    got = block.block_norm_backward(c.x, c.b, stats, c.dy, c.dh, **c.kw)
    ref = backward64(c)
    assert set(ref) >= {"dx", "dbranch", "dpost_weight", "dpre_weight"} and (c.g is None) == ("dgate" not in ref)
    for name, (r, mag) in ref.items():
        near((name, T, D, mode), getattr(got, name), r, mag, OPS + T)


@pytest.mark.parametrize("mode", ["none", "channel", "token", "full"])
@pytest.mark.parametrize("res", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,D", SHAPES)
def test_many_rows_a_group(T, D, res, mode):
    assert T > groups_at_most()
    check(Case(T, D, res, torch.float32 if mode != "channel" else torch.bfloat16, mode, 1, 1, pad=0 if T % 2 else 8, seed=T), T, D, mode)


# (gate rows): one (partial sums over slabs of many rows), a few, one for two
# rows (more than there are groups: several whole gate rows a group)
@pytest.mark.parametrize("T,D,groups", [(4000, 1411, 1), (4000, 1411, 5), (3000, 2056, 4), (3000, 2056, 1500), (2500, 7168, 2),
                                        (2500, 7168, 500), (9000, 24, 3), (9000, 24, 4500), (4000, 1411, 1000), (7200, 1024, 3600),
                                        (2460, 8191, 820)])
@pytest.mark.parametrize("res", [torch.bfloat16, torch.float32])
def test_grouped_gates(T, D, groups, res):
    assert T > groups_at_most()
    check(Case(T, D, res, torch.float32 if groups % 2 else torch.bfloat16, "group", 1, 1, pad=0 if groups % 2 else 8, seed=groups,
               groups=groups), T, D, "group")


@pytest.mark.parametrize("D", [1411, 2056, 7168])
def test_in_place_over_many_rows(D):
    from mixture_experts_routed_route_gb300 import block
    T = 2600
    assert T > groups_at_most()
    c = Case(T, D, torch.bfloat16, torch.bfloat16, "channel", 1, 1, seed=1)
    y, h = block.block_norm(c.x, c.b, eps=c.eps, **c.kw)
    x, b = c.x.clone(), c.b.clone()
    y1, h1 = block.block_norm(x, b, eps=c.eps, y=x, h=b, **c.kw)
    assert y1 is x and h1 is b and torch.equal(x, y) and torch.equal(b, h)
