"""The cross entropy without a GPU: the struct's layout and the refusals, which come before any CUDA call."""

import ctypes

import pytest
import torch

from mixture_experts_routed_route_gb300 import abi, loss

BAD, UNSUPPORTED = abi.MOE_ERR_INVALID_ARG, abi.MOE_ERR_UNSUPPORTED


def cfg(**kw):
    c = abi.moe_linear_ce_config(4, 64, 100, 8, 1.0, 0.0, -100, 0)
    for k, v in kw.items():
        setattr(c, k, v)
    return c


def forward(c, h=16, weight=16, targets=16, loss=16, lse=16, ws=256, nb=1 << 40, err=4):
    return abi.LIB.moe_linear_ce_forward(None if c is None else ctypes.byref(c), h, weight, targets, loss, lse, ws, nb, err,
                                         None)


def backward(c, h=16, weight=16, targets=16, lse=16, d_loss=16, dh=16, dweight=16, ws=256, nb=1 << 40, err=4):
    return abi.LIB.moe_linear_ce_backward(None if c is None else ctypes.byref(c), h, weight, targets, lse, d_loss, dh,
                                          dweight, ws, nb, err, None)


def test_struct_layout():
    assert ctypes.sizeof(abi.moe_linear_ce_config) == 4 * 4 + 2 * 4 + 2 * 8
    assert abi.moe_linear_ce_config.ignore_index.offset == 24


@pytest.mark.parametrize("fields,status", [
    (dict(tokens=-1), BAD), (dict(d_model=0), BAD), (dict(vocab=0), BAD), (dict(target_bytes=2), BAD),
    (dict(logit_scale=0.0), BAD), (dict(logit_scale=-1.0), BAD), (dict(logit_scale=float("nan")), BAD),
    (dict(logit_scale=float("inf")), BAD), (dict(z_weight=-1e-4), BAD), (dict(z_weight=float("inf")), BAD),
    (dict(z_weight=float("nan")), BAD), (dict(h_stride=63), BAD), (dict(h_stride=-64), BAD),
    (dict(d_model=63), UNSUPPORTED), (dict(d_model=65544), UNSUPPORTED), (dict(vocab=(1 << 24) + 1), UNSUPPORTED),
    (dict(tokens=(1 << 24) + 1), UNSUPPORTED), (dict(tokens=1 << 24, vocab=1 << 23), UNSUPPORTED)])
def test_refuses_configs(fields, status):
    c = cfg(**fields)
    assert forward(c) == status
    assert backward(c) == status
    assert abi.moe_linear_ce_workspace_bytes(c, 1, 256) == 0


def test_refuses_pointers():
    assert forward(None) == backward(None) == BAD
    for name in ("h", "weight", "targets", "lse"):
        for v in (None, 24):
            assert forward(cfg(), **{name: v}) == backward(cfg(), **{name: v}) == BAD, (name, v)
    for kw in (dict(loss=None), dict(loss=24), dict(ws=None), dict(ws=16), dict(err=None), dict(err=6)):
        assert forward(cfg(), **kw) == BAD, kw
    for kw in (dict(d_loss=None), dict(d_loss=24), dict(dh=24), dict(dweight=24), dict(dh=None, dweight=None), dict(ws=None),
               dict(ws=16), dict(err=None), dict(err=6)):
        assert backward(cfg(), **kw) == BAD, kw
    assert forward(cfg(tokens=0), None, None, None, None, None, None, 0, None) == abi.MOE_OK
    assert backward(cfg(tokens=0), None, None, None, None, None, None, None, None, 0, None) == abi.MOE_OK
    assert backward(cfg(tokens=0), dweight=24) == BAD
    for piece in (0, -1):
        assert abi.moe_linear_ce_workspace_bytes(cfg(), 1, piece) == 0


def test_wrapper_refusals():
    h, w, t = torch.zeros(4, 64).bfloat16(), torch.zeros(9, 64).bfloat16(), torch.zeros(4, dtype=torch.int64)
    with pytest.raises(ValueError):
        loss.linear_cross_entropy(h, w, t)          # host tensors
    c = cfg()
    for piece in (0, 1 << 31):
        with pytest.raises(ValueError):
            loss._workspace_bytes(c, True, piece)
