"""What a transformer block runs around the routed layer, on torch tensors:
the norms before and after a block with its gate and scaled residual
(``block_norm``), and the router's choice of experts with its scores
(``topk_gate``), each with its backward.

Argument checks and buffers are here; every computation runs in the CUDA
library (``moe_block_norm_*`` and ``moe_topk_gate_*`` of the C ABI).  Calls
enqueue on the current stream of the inputs' device, or on ``stream`` (a torch
stream or a raw handle); buffers that a call makes are allocated on the stream
it runs on.  Inputs that another stream still writes are the caller's to
order, as with any torch operator.
"""

from typing import NamedTuple, Optional

import torch

from . import abi

_TYPE = {torch.bfloat16: abi.MOE_TYPE_BF16, torch.float32: abi.MOE_TYPE_FP32}
_SCORE = {"softmax": abi.MOE_SCORE_SOFTMAX, "sigmoid": abi.MOE_SCORE_SIGMOID}


def on_stream(fn, device, stream):
    """fn() with `device` current and `stream` (None: the current one) as its stream."""
    if stream is None and device.index == torch.cuda.current_device():
        return fn()
    with torch.cuda.device(device):
        if stream is None:
            return fn()
        if isinstance(stream, int):
            stream = torch.cuda.ExternalStream(stream, device=device)
        with torch.cuda.stream(stream):
            return fn()


def _need(ok, message):
    if not ok:
        raise ValueError(message)


def _rows(name, t, dtype, shape, device):
    """A [T, D] tensor whose rows are contiguous; its row stride."""
    _need(t.dtype == dtype and tuple(t.shape) == shape and t.device == device,
          f"{name}: expected {dtype} {list(shape)} on {device}, got {t.dtype} {list(t.shape)} on {t.device}")
    T, D = shape
    if T <= 1:
        _need(D <= 1 or T == 0 or t.stride(1) == 1, f"{name}: its columns are not contiguous")
        return D
    _need(D == 1 or t.stride(1) == 1, f"{name}: its columns are not contiguous")
    _need(t.stride(0) >= D, f"{name}: its rows overlap (stride {t.stride(0)} for {D} columns)")
    return t.stride(0)


def _dense(name, t, dtype, shape, device):
    _need(t.dtype == dtype and tuple(t.shape) == shape and t.device == device and t.is_contiguous(),
          f"{name}: expected contiguous {dtype} {list(shape)} on {device}, got {t.dtype} {list(t.shape)} on {t.device}")


class _Norm:
    """The checked arguments shared by block_norm and its backward."""

    def __init__(self, x, branch, gate, post_weight, pre_weight, residual_scale, branch_scale, eps, weight_offset):
        _need(x.dim() == 2 and x.is_cuda and x.dtype in _TYPE, "x: expected a CUDA bfloat16 or float32 [T, D] tensor")
        T, D = self.shape = tuple(x.shape)
        dev = self.device = x.device
        cfg = self.cfg = abi.moe_block_norm_config(T, D, _TYPE[x.dtype], 0, 0, abi.MOE_GATE_NONE, 0, residual_scale,
                                                   branch_scale, eps, weight_offset, 0, 0, 0, 0)
        cfg.x_stride = _rows("x", x, x.dtype, self.shape, dev)
        if branch is not None:
            cfg.branch_stride = _rows("branch", branch, torch.bfloat16, self.shape, dev)
        else:
            _need(gate is None and post_weight is None, "a gate or post_weight needs a branch")
        weights = [w for w in (post_weight, pre_weight) if w is not None]
        for w in weights:
            _need(w.dtype in _TYPE, "weights are bfloat16 or float32")
            _dense("weight", w, weights[0].dtype, (D,), dev)
            cfg.weight_type = _TYPE[w.dtype]
        if gate is not None:
            _need(gate.dtype in _TYPE and gate.device == dev and gate.is_contiguous() and gate.dim() in (1, 2),
                  f"gate: expected contiguous bfloat16 or float32 [D], [G, D] or [T, 1] on {dev}")
            cfg.gate_type = _TYPE[gate.dtype]
            if gate.dim() == 1 and gate.shape[0] == D:
                cfg.gate_mode = abi.MOE_GATE_CHANNEL
            elif gate.dim() == 2 and gate.shape[1] == D and gate.shape[0] > 0 and T % gate.shape[0] == 0:
                cfg.gate_mode, cfg.gate_rows = abi.MOE_GATE_GROUP, gate.shape[0]
            elif gate.dim() == 2 and tuple(gate.shape) == (T, 1):
                cfg.gate_mode = abi.MOE_GATE_TOKEN
            else:
                raise ValueError(f"gate {list(gate.shape)}: expected [{D}], [G, {D}] with G dividing {T}, or [{T}, 1]")


def block_norm(x, branch=None, *, gate=None, post_weight=None, pre_weight=None, residual_scale=1.0, branch_scale=1.0,
               eps=1e-6, weight_offset=0.0, y=None, h=None, stats=None, stream=None):
    """(y, h) of one block boundary:

        y = residual_scale * x + branch_scale * gate * rms_norm(branch) * (post_weight + weight_offset)
        h = rms_norm(y) * (pre_weight + weight_offset)

    x: [T, D] bfloat16 or float32; branch: [T, D] bfloat16 or None (a norm
    alone: y is then x, and is written only where a ``y`` is given or the
    residual is scaled).  post_weight None: no norm after the block;
    pre_weight None: no h (None is returned in its place).  gate: [D] (a
    channel), [G, D] (row t takes gate row t // (T / G)) or [T, 1] (a token).
    ``y`` may be x and ``h`` may be branch (in place).  ``stats``: a float32
    [2, T] tensor for the backward to read."""
    n = _Norm(x, branch, gate, post_weight, pre_weight, residual_scale, branch_scale, eps, weight_offset)
    cfg, dev = n.cfg, n.device
    if y is not None:
        cfg.y_stride = _rows("y", y, x.dtype, n.shape, dev)
    if h is not None:
        _need(pre_weight is not None, "h needs a pre_weight")
        cfg.h_stride = _rows("h", h, torch.bfloat16, n.shape, dev)
    if stats is not None:
        _dense("stats", stats, torch.float32, (2, n.shape[0]), dev)
    _need(branch is not None or pre_weight is not None or y is not None or residual_scale != 1.0,
          "nothing to compute: no branch, no pre_weight")
    same = branch is None and y is None and residual_scale == 1.0

    def run():
        yy = y if y is not None or same else torch.empty(n.shape, dtype=x.dtype, device=dev)
        hh = h if h is not None or pre_weight is None else torch.empty(n.shape, dtype=torch.bfloat16, device=dev)
        abi.moe_block_norm_forward(cfg, x, branch, gate, post_weight, pre_weight, yy, hh, stats)
        return (x if same else yy), hh

    return on_stream(run, dev, stream)


class BlockNormGrads(NamedTuple):
    dx: torch.Tensor
    dbranch: Optional[torch.Tensor]
    dgate: Optional[torch.Tensor]
    dpost_weight: Optional[torch.Tensor]
    dpre_weight: Optional[torch.Tensor]


def block_norm_backward(x, branch, stats, dy, dh=None, *, gate=None, post_weight=None, pre_weight=None,
                        residual_scale=1.0, branch_scale=1.0, weight_offset=0.0, stream=None):
    """Gradients (BlockNormGrads) of block_norm's inputs from ``dy`` (x's
    type; None: zero) and ``dh`` (bfloat16; given with pre_weight), with the
    forward's inputs and ``stats``.  dx has x's type, dbranch is bfloat16,
    dgate has the gate's shape and type, the weights' gradients are float32."""
    n = _Norm(x, branch, gate, post_weight, pre_weight, residual_scale, branch_scale, 1.0, weight_offset)
    cfg, dev = n.cfg, n.device
    T, D = n.shape
    _need((dh is not None) == (pre_weight is not None), "dh goes with pre_weight")
    _need(dy is not None or dh is not None, "no gradient given")
    if dy is not None:
        cfg.y_stride = _rows("dy", dy, x.dtype, n.shape, dev)
    if dh is not None:
        cfg.h_stride = _rows("dh", dh, torch.bfloat16, n.shape, dev)
    if post_weight is not None or pre_weight is not None:
        _need(stats is not None, "the norms' backward needs the forward's stats")
        _dense("stats", stats, torch.float32, (2, T), dev)

    def run():
        dx = torch.empty(n.shape, dtype=x.dtype, device=dev)
        dbranch = None if branch is None else torch.empty(n.shape, dtype=torch.bfloat16, device=dev)
        dgate = None if gate is None else torch.empty_like(gate)
        dpost = None if post_weight is None else torch.empty(D, dtype=torch.float32, device=dev)
        dpre = None if pre_weight is None else torch.empty(D, dtype=torch.float32, device=dev)
        nb = abi.moe_block_norm_workspace_bytes(cfg)
        ws = torch.empty(nb, dtype=torch.uint8, device=dev)
        abi.moe_block_norm_backward(cfg, x, branch, gate, post_weight, pre_weight, stats, dy, dh, dx, dbranch, dgate,
                                    dpost, dpre, ws, nb)
        return BlockNormGrads(dx, dbranch, dgate, dpost, dpre)

    return on_stream(run, dev, stream)


def _gate_config(logits, top_k, score, renormalize, scale):
    _need(logits.dim() == 2 and logits.is_cuda and logits.dtype in _TYPE,
          "logits: expected a CUDA bfloat16 or float32 [T, E] tensor")
    _need(score in _SCORE, f"score: one of {sorted(_SCORE)}")
    T, E = logits.shape
    cfg = abi.moe_topk_gate_config(T, E, top_k, _TYPE[logits.dtype], _SCORE[score], 1 if renormalize else 0, scale, 0)
    cfg.logits_stride = _rows("logits", logits, logits.dtype, (T, E), logits.device)
    return cfg


def topk_gate(logits, top_k, *, score="softmax", renormalize=False, scale=1.0, select_bias=None, ids=None, scores=None,
              stream=None):
    """(ids int32 [T, top_k], scores float32 [T, top_k]) of router logits
    [T, E] (bfloat16 or float32), as MoELayer.forward takes them: the top_k
    largest logits (+ select_bias [E] float32, for the choice only), equal
    ones by index; masked experts (-inf) are never chosen, and places without
    an expert are inactive routes (id -1, score 0).  score: "softmax" over
    all experts or "sigmoid"; renormalize: over the chosen ones; times scale."""
    cfg = _gate_config(logits, top_k, score, renormalize, scale)
    dev, shape = logits.device, (logits.shape[0], top_k)
    if select_bias is not None:
        _dense("select_bias", select_bias, torch.float32, (logits.shape[1],), dev)
    if ids is not None:
        _dense("ids", ids, torch.int32, shape, dev)
    if scores is not None:
        _dense("scores", scores, torch.float32, shape, dev)

    def run():
        i = torch.empty(shape, dtype=torch.int32, device=dev) if ids is None else ids
        s = torch.empty(shape, dtype=torch.float32, device=dev) if scores is None else scores
        abi.moe_topk_gate_forward(cfg, logits, select_bias, i, s)
        return i, s

    return on_stream(run, dev, stream)


def topk_gate_backward(logits, ids, d_scores, *, score="softmax", renormalize=False, scale=1.0, d_logits=None,
                       stream=None):
    """The gradient [T, E] of the logits (their type) from d_scores [T, top_k]
    (float32, MoELayer.backward's) at topk_gate's ids."""
    _need(ids.dim() == 2, "ids: expected [T, top_k]")
    cfg = _gate_config(logits, ids.shape[1], score, renormalize, scale)
    dev, shape = logits.device, (logits.shape[0], ids.shape[1])
    _dense("ids", ids, torch.int32, shape, dev)
    _dense("d_scores", d_scores, torch.float32, shape, dev)
    if d_logits is not None:
        _dense("d_logits", d_logits, logits.dtype, tuple(logits.shape), dev)

    def run():
        d = torch.empty(logits.shape, dtype=logits.dtype, device=dev) if d_logits is None else d_logits
        abi.moe_topk_gate_backward(cfg, logits, ids, d_scores, d)
        return d

    return on_stream(run, dev, stream)
