"""Calls around the routed layer that need no GPU: the structs' layouts, the
sizes computed on the host, and the refusals, which come before any CUDA call
(a refused call would otherwise fail here for want of a device)."""

import ctypes

import pytest
import torch

from mixture_experts_routed_route_gb300 import abi


def norm_cfg(**kw):
    c = abi.moe_block_norm_config(4, 64, abi.MOE_TYPE_BF16, abi.MOE_TYPE_BF16, abi.MOE_TYPE_BF16, abi.MOE_GATE_NONE, 0,
                                  1.0, 1.0, 1e-6, 0.0, 0, 0, 0, 0)
    for k, v in kw.items():
        setattr(c, k, v)
    return c


def norm_forward(c, x=16, branch=None, gate=None, post=None, pre=16, y=None, h=16, stats=None):
    return abi.LIB.moe_block_norm_forward(None if c is None else ctypes.byref(c), x, branch, gate, post, pre, y, h, stats,
                                          None)


def test_struct_layouts():
    assert ctypes.sizeof(abi.moe_block_norm_config) == 11 * 4 + 4 + 4 * 8
    assert abi.moe_block_norm_config.x_stride.offset == 48
    assert ctypes.sizeof(abi.moe_topk_gate_config) == 7 * 4 + 4 + 8
    assert ctypes.sizeof(abi.moe_muon_config) == 4 * 4 + abi.MOE_MUON_MAX_STEPS * 12 + 4
    assert ctypes.sizeof(abi.moe_muon_rates) == 5 * 4


def test_block_norm_accepts_no_rows():
    assert norm_forward(norm_cfg(tokens=0)) == abi.MOE_OK


@pytest.mark.parametrize("fields", [
    dict(tokens=-1), dict(d_model=0), dict(residual_type=2), dict(weight_type=7), dict(gate_type=-1), dict(gate_mode=4),
    dict(eps=0.0), dict(eps=-1.0), dict(eps=float("nan")), dict(eps=float("inf")), dict(residual_scale=float("nan")),
    dict(branch_scale=float("inf")), dict(weight_offset=float("nan")), dict(x_stride=63), dict(h_stride=-64),
    dict(y_stride=1), dict(branch_stride=32)])
def test_block_norm_refuses_configs(fields):
    assert norm_forward(norm_cfg(**fields)) == abi.MOE_ERR_INVALID_ARG


def test_block_norm_refuses_parts_that_do_not_belong_together():
    bad = abi.MOE_ERR_INVALID_ARG
    assert norm_forward(None) == bad
    assert norm_forward(norm_cfg(), x=None) == bad
    assert norm_forward(norm_cfg(), post=16) == bad                       # a weight after no block
    assert norm_forward(norm_cfg(), gate=16) == bad                       # a gate of no block
    assert norm_forward(norm_cfg(gate_mode=abi.MOE_GATE_CHANNEL), branch=16) == bad   # a mode without a gate
    assert norm_forward(norm_cfg(), branch=16, gate=16) == bad            # a gate without a mode
    assert norm_forward(norm_cfg(), h=None) == bad                        # a norm without its output
    assert norm_forward(norm_cfg(), pre=None) == bad                      # an output without its norm
    assert norm_forward(norm_cfg(), pre=None, h=None) == bad              # nothing to write
    assert norm_forward(norm_cfg(gate_mode=abi.MOE_GATE_GROUP, gate_rows=3), branch=16, gate=16) == bad   # 4 rows by 3
    assert norm_forward(norm_cfg(gate_mode=abi.MOE_GATE_GROUP, gate_rows=0), branch=16, gate=16) == bad
    for name in ("x", "pre", "h"):
        assert norm_forward(norm_cfg(), **{name: 24}) == bad              # not 16-byte aligned
    assert norm_forward(norm_cfg(d_model=8193)) == abi.MOE_ERR_UNSUPPORTED


def norm_backward(c, x=16, branch=16, gate=None, post=16, pre=16, stats=16, dy=16, dh=16, dx=16, dbranch=16, dgate=None,
                  dpost=16, dpre=16, ws=16, nb=1 << 30):
    return abi.LIB.moe_block_norm_backward(ctypes.byref(c), x, branch, gate, post, pre, stats, dy, dh, dx, dbranch, dgate,
                                           dpost, dpre, ws, nb, None)


def test_block_norm_backward_refusals():
    bad = abi.MOE_ERR_INVALID_ARG
    c = norm_cfg()
    assert norm_backward(c, dh=None) == bad
    assert norm_backward(c, dy=None, dh=None, pre=None, dpre=None) == bad
    assert norm_backward(c, dbranch=None) == bad
    assert norm_backward(c, branch=None) == bad
    assert norm_backward(c, dpost=None) == bad
    assert norm_backward(c, dpre=None) == bad
    assert norm_backward(c, dgate=16) == bad
    assert norm_backward(c, stats=None) == bad
    assert norm_backward(c, dx=8) == bad
    assert norm_backward(norm_cfg(d_model=9000)) == abi.MOE_ERR_UNSUPPORTED


def gate_cfg(**kw):
    c = abi.moe_topk_gate_config(4, 8, 2, abi.MOE_TYPE_FP32, abi.MOE_SCORE_SOFTMAX, 0, 1.0, 0)
    for k, v in kw.items():
        setattr(c, k, v)
    return c


@pytest.mark.parametrize("fields", [
    dict(tokens=-1), dict(num_experts=0), dict(num_experts=1025), dict(top_k=0), dict(top_k=9),
    dict(num_experts=64, top_k=33), dict(logits_type=2), dict(score=2), dict(scale=float("nan")), dict(logits_stride=7),
    dict(logits_stride=-8)])
def test_topk_gate_refuses_configs(fields):
    c = gate_cfg(**fields)
    assert abi.LIB.moe_topk_gate_forward(ctypes.byref(c), 16, None, 16, 16, None) == abi.MOE_ERR_INVALID_ARG
    assert abi.LIB.moe_topk_gate_backward(ctypes.byref(c), 16, 16, 16, 16, None) == abi.MOE_ERR_INVALID_ARG


def test_topk_gate_refuses_pointers():
    c = ctypes.byref(gate_cfg())
    fwd, bwd, bad = abi.LIB.moe_topk_gate_forward, abi.LIB.moe_topk_gate_backward, abi.MOE_ERR_INVALID_ARG
    assert fwd(None, 16, None, 16, 16, None) == bad
    for args in ((None, None, 16, 16), (16, None, None, 16), (16, None, 16, None), (20, None, 16, 16), (16, 20, 16, 16),
                 (16, None, 20, 16), (16, None, 16, 20)):
        assert fwd(c, *args, None) == bad, args
    for args in ((None, 16, 16, 16), (16, None, 16, 16), (16, 16, None, 16), (16, 16, 16, None), (16, 16, 16, 18)):
        assert bwd(c, *args, None) == bad, args
    assert fwd(ctypes.byref(gate_cfg(tokens=0)), None, None, None, None, None) == abi.MOE_OK


def muon_cfg(**kw):
    c = abi.moe_muon_config(2, 64, 96, 5)
    c.eps = 1e-7
    for s in range(5):
        c.coefficients[s][:] = (3.4445, -4.7750, 2.0315)
    for k, v in kw.items():
        setattr(c, k, v)
    return c


def test_muon_workspace_grows_by_matrices():
    c = muon_cfg()
    one, two = abi.moe_muon_workspace_bytes(c, 1), abi.moe_muon_workspace_bytes(c, 2)
    # X in halves (hi twice, lo twice for sizes up to 256), A and B, B's diagonal
    assert two - one >= 64 * 128 * 2 * 4 + 2 * 64 * 64 * 2 + 64 * 4
    assert abi.moe_muon_workspace_bytes(c, 5) - two == 3 * (two - one)
    assert abi.moe_muon_workspace_bytes(muon_cfg(steps=16), 2) == two     # one workspace serves any number of steps
    tall = muon_cfg(rows=96, cols=64)
    assert abi.moe_muon_workspace_bytes(tall, 1) > 0


@pytest.mark.parametrize("fields", [dict(batch=-1), dict(rows=0), dict(cols=0), dict(steps=0), dict(steps=17),
                                    dict(eps=0.0), dict(eps=float("nan"))])
def test_muon_refuses_configs(fields):
    c = muon_cfg(**fields)
    bad = abi.MOE_ERR_INVALID_ARG
    assert abi.LIB.moe_orthogonalize(ctypes.byref(c), 16, 0, 16, 256, 1 << 30, 4, None) == bad
    assert abi.moe_muon_workspace_bytes(c, 1) == 0


def test_muon_refusals():
    bad = abi.MOE_ERR_INVALID_ARG
    c = muon_cfg()
    p = ctypes.byref(c)
    orth = abi.LIB.moe_orthogonalize
    assert orth(None, 16, 0, 16, 256, 1 << 30, 4, None) == bad
    for args in ((None, 0, 16, 256, 4), (16, 2, 16, 256, 4), (16, 0, None, 256, 4), (16, 0, 16, None, 4),
                 (16, 0, 16, 256, None), (24, 0, 16, 256, 4), (16, 0, 24, 256, 4), (16, 0, 16, 272, 4), (16, 0, 16, 256, 5)):
        x, t, o, w, e = args
        assert orth(p, x, t, o, w, 1 << 30, e, None) == bad, args
    assert orth(p, 16, 0, 16, 256, abi.moe_muon_workspace_bytes(c, 1) - 1, 4, None) == abi.MOE_ERR_CAPACITY
    assert orth(ctypes.byref(muon_cfg(rows=65537)), 16, 0, 16, 256, 1 << 30, 4, None) == abi.MOE_ERR_UNSUPPORTED
    assert orth(ctypes.byref(muon_cfg(batch=0)), None, 0, None, None, 0, None, None) == abi.MOE_OK
    big = muon_cfg()
    big.coefficients[2][1] = 17.0
    assert orth(ctypes.byref(big), 16, 0, 16, 256, 1 << 30, 4, None) == bad
    upd = abi.LIB.moe_muon_update
    rates = abi.moe_muon_rates(1e-3, 0.95, 0.1, 1.0, 1)
    good = dict(weight=16, wt=1, grad=16, gt=0, mom=16, copy=None, ws=256, err=4)

    def call(rates=rates, **kw):
        a = dict(good, **kw)
        return upd(p, None if rates is None else ctypes.byref(rates), a["weight"], a["wt"], a["grad"], a["gt"], a["mom"],
                   a["copy"], a["ws"], 0, a["err"], None)

    assert call() == abi.MOE_ERR_CAPACITY                                # all but the workspace's size is fine
    for kw in (dict(weight=None), dict(grad=None), dict(mom=None), dict(ws=None), dict(err=None), dict(wt=2), dict(gt=3),
               dict(weight=8), dict(grad=8), dict(mom=8), dict(copy=8), dict(wt=0, copy=16)):
        assert call(**kw) == bad, kw
    assert call(rates=None) == bad
    for i in range(4):
        r = [1e-3, 0.95, 0.1, 1.0]
        r[i] = float("inf")
        assert call(rates=abi.moe_muon_rates(*r, 1)) == bad


def test_wrappers_refuse_host_tensors():
    from mixture_experts_routed_route_gb300 import block, optim
    x = torch.zeros(4, 64)
    with pytest.raises(ValueError):
        block.block_norm(x, pre_weight=torch.ones(64))
    with pytest.raises(ValueError):
        block.topk_gate(x, 2)
    with pytest.raises(ValueError):
        optim.orthogonalize(torch.zeros(2, 4, 4))
    with pytest.raises(ValueError):
        optim._config((2, 4), 5, optim.COEFFICIENTS, 1e-7)
    with pytest.raises(ValueError):
        optim._config((2, 4, 4), 5, [(1.0, 0.0, 0.0)] * 3, 1e-7)
