"""Dropout and layer norm without a GPU: the generator's published vectors,
the structs' layouts and the refusals, which come before any CUDA call."""

import ctypes

import pytest
import torch

import dropout_oracle as oracle
from mixture_experts_routed_route_gb300 import abi, block

BAD = abi.MOE_ERR_INVALID_ARG


def test_generator_against_published_vectors():
    """Known answers of Philox4x32-10 for zeros, ones and the digits of pi."""
    cases = [((0, 0, 0, 0), (0, 0), (0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8)),
             ((0xFFFFFFFF,) * 4, (0xFFFFFFFF,) * 2, (0x408F276D, 0x41C83B0E, 0xA20BC7C6, 0x6D5451FD)),
             ((0x243F6A88, 0x85A308D3, 0x13198A2E, 0x03707344), (0xA4093822, 0x299F31D0),
              (0xD16CFE09, 0x94FDCCEB, 0x5001E420, 0x24126EA1))]
    for counter, key, want in cases:
        assert tuple(int(w) for w in oracle.philox(counter, key)) == want


def test_mask_statistics():
    """Shares of kept elements are within five standard deviations, and masks of other steps, sites and seeds differ."""
    n = 1 << 18
    k, f = oracle.keep(512, 512, 0.25, 7, 3, 1)
    assert abs(float(k.double().mean()) - 0.75) < 5 * (0.75 * 0.25 / n) ** 0.5
    assert f == 65536 / 49152
    for other in (oracle.keep(512, 512, 0.25, 8, 3, 1), oracle.keep(512, 512, 0.25, 7, 4, 1),
                  oracle.keep(512, 512, 0.25, 7, 3, 2)):
        agree = float((k == other[0]).double().mean())        # 0.75^2 + 0.25^2 of independent ones
        assert abs(agree - 0.625) < 5 * (0.625 * 0.375 / n) ** 0.5


def test_struct_layouts():
    assert ctypes.sizeof(abi.moe_dropout_config) == 4 * 4 + 8 + 3 * 8
    assert abi.moe_dropout_config.p.offset == 16
    assert ctypes.sizeof(abi.moe_layer_norm_config) == 8 * 4 + 8 + 4 * 8
    assert abi.moe_layer_norm_config.dropout.offset == 32


def drop_cfg(**kw):
    c = abi.moe_dropout_config(4, 64, abi.MOE_TYPE_BF16, 0, 0.1, 0, 0, 0)
    for k, v in kw.items():
        setattr(c, k, v)
    return c


def drop(c, x=16, residual=None, rng=16, out=16):
    return abi.LIB.moe_dropout(None if c is None else ctypes.byref(c), x, residual, rng, out, None)


@pytest.mark.parametrize("fields", [dict(tokens=-1), dict(d_model=0), dict(type=2), dict(p=-0.1), dict(p=1.01),
                                    dict(p=float("nan")), dict(x_stride=63), dict(out_stride=-64), dict(residual_stride=1)])
def test_dropout_refuses_configs(fields):
    assert drop(drop_cfg(**fields)) == BAD


def test_dropout_refuses_pointers():
    assert drop(None) == BAD
    for kw in (dict(x=None), dict(out=None), dict(rng=None), dict(x=24), dict(residual=24), dict(rng=24), dict(out=24)):
        assert drop(drop_cfg(), **kw) == BAD, kw
    assert drop(drop_cfg(tokens=0), None, None, None, None) == abi.MOE_OK


def norm_cfg(**kw):
    c = abi.moe_layer_norm_config(4, 64, abi.MOE_TYPE_BF16, abi.MOE_TYPE_BF16, 1.0, 1.0, 1e-5, 0, 0.0, 0, 0, 0, 0)
    for k, v in kw.items():
        setattr(c, k, v)
    return c


def norm(c, x=16, branch=16, weight=16, bias=16, rng=16, y=16, h=16, stats=16):
    return abi.LIB.moe_layer_norm_forward(None if c is None else ctypes.byref(c), x, branch, weight, bias, rng, y, h, stats,
                                          None)


def norm_back(c, y=16, weight=16, stats=16, rng=16, dy=16, dh=16, dx=16, dbranch=16, dweight=16, dbias=16, ws=16,
              nb=1 << 30):
    return abi.LIB.moe_layer_norm_backward(None if c is None else ctypes.byref(c), y, weight, stats, rng, dy, dh, dx,
                                           dbranch, dweight, dbias, ws, nb, None)


@pytest.mark.parametrize("fields", [
    dict(tokens=-1), dict(d_model=0), dict(residual_type=2), dict(weight_type=-1), dict(eps=0.0), dict(eps=float("nan")),
    dict(eps=float("inf")), dict(residual_scale=float("inf")), dict(branch_scale=float("nan")), dict(dropout=1.5),
    dict(dropout=-0.1), dict(dropout=float("nan")), dict(x_stride=63), dict(branch_stride=32), dict(y_stride=-64),
    dict(h_stride=1)])
def test_layer_norm_refuses_configs(fields):
    c = norm_cfg(**fields)
    assert norm(c) == BAD
    assert norm_back(c) == BAD
    assert abi.moe_layer_norm_workspace_bytes(c) == 0


def test_layer_norm_refuses_pointers():
    assert norm(None) == BAD and norm_back(None) == BAD
    for kw in (dict(x=None), dict(h=None), dict(x=24), dict(branch=24), dict(weight=24), dict(bias=24), dict(rng=24),
               dict(y=24), dict(h=24), dict(stats=24)):
        assert norm(norm_cfg(), **kw) == BAD, kw
    for kw in (dict(rng=None), dict(branch=None)):
        assert norm(norm_cfg(dropout=0.1), **kw) == BAD, kw
    for kw in (dict(y=None), dict(stats=None), dict(dh=None), dict(dx=None, dbranch=None, dweight=None, dbias=None),
               dict(y=24), dict(weight=24), dict(stats=24), dict(rng=24), dict(dy=24), dict(dh=24), dict(dx=24),
               dict(dbranch=24), dict(dweight=24), dict(dbias=24), dict(ws=24)):
        assert norm_back(norm_cfg(), **kw) == BAD, kw
    for kw in (dict(rng=None), dict(dbranch=None)):
        assert norm_back(norm_cfg(dropout=0.1), **kw) == BAD, kw
    assert norm(norm_cfg(d_model=8193)) == norm_back(norm_cfg(d_model=8193)) == abi.MOE_ERR_UNSUPPORTED
    assert norm(norm_cfg(tokens=0), None, None, None, None, None, None, None, None) == abi.MOE_OK


def test_wrappers_refuse_host_tensors_and_bad_probabilities():
    x, rng = torch.zeros(4, 64), torch.zeros(2, dtype=torch.int64)
    with pytest.raises(ValueError):
        block.dropout(x, 0.1, rng)
    with pytest.raises(ValueError):
        block.layer_norm(x)
    for p in (-0.5, 1.5, float("nan")):
        with pytest.raises(ValueError):
            block._check_rng(p, rng, 0, rng.device)
    with pytest.raises(ValueError):
        block._check_rng(0.5, None, 0, rng.device)
    with pytest.raises(ValueError):
        block._check_rng(0.5, rng.to(torch.int32), 0, rng.device)
    for site in (-1, 1 << 32):
        with pytest.raises(ValueError):
            block._check_rng(0.5, rng, site, rng.device)
    block._check_rng(0.0, None, 0, rng.device)
