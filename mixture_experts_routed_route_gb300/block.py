"""What a transformer block runs around the routed layer, on torch tensors:
the norms before and after a block with its gate and scaled residual
(``block_norm``), layer norm with the scaled residual and dropout on the branch
(``layer_norm``), dropout alone (``dropout``), and the router's choice of
experts with its scores (``topk_gate``), each with its backward.

Argument checks and buffers are here; every computation runs in the CUDA
library (``moe_block_norm_*``, ``moe_layer_norm_*``, ``moe_dropout`` and
``moe_topk_gate_*`` of the C ABI).  Calls
enqueue on the current stream of the inputs' device, or on ``stream`` (a torch
stream or a raw handle); buffers that a call makes are allocated on the stream
it runs on.  Inputs that another stream still writes are the caller's to
order, as with any torch operator.  The library wants tensors that start at a
16-byte boundary; where one does not (a slice of tokens of an odd width, a view
into a flat buffer), the call works on an aligned copy of it and copies results
back, one more pass over that tensor.
"""

import ctypes
from typing import NamedTuple, Optional

import torch

from . import abi

_TYPE = {torch.bfloat16: abi.MOE_TYPE_BF16, torch.float32: abi.MOE_TYPE_FP32}
_NormConfig, _GateConfig = abi.moe_block_norm_config, abi.moe_topk_gate_config
_LayerNormConfig, _DropoutConfig = abi.moe_layer_norm_config, abi.moe_dropout_config
_SCORE = {"softmax": abi.MOE_SCORE_SOFTMAX, "sigmoid": abi.MOE_SCORE_SIGMOID}


# sizes are int32 in the C structs
_MOST = 1 << 31

# the raw handle of a device's current stream (torch.cuda.current_stream builds a Stream object each time)
_raw_stream = torch._C._cuda_getCurrentRawStream
_current_device = torch.cuda.current_device
_BF16, _FP32, _INT32, _INT64 = torch.bfloat16, torch.float32, torch.int32, torch.int64
_empty, _empty_like, _byref = torch.empty, torch.empty_like, ctypes.byref
_LIB, _INVALID = abi.LIB, abi.MOE_ERR_INVALID_ARG


def on_stream(fn, device, stream):
    """fn(raw stream) with `device` current, on `stream` (None: the current one), which is then current too."""
    if stream is None and device.index == _current_device():
        return fn(_raw_stream(device.index))
    with torch.cuda.device(device):
        if stream is None:
            return fn(_raw_stream(device.index))
        if isinstance(stream, int):
            stream = torch.cuda.ExternalStream(stream, device=device)
        with torch.cuda.stream(stream):
            return fn(stream.cuda_stream)


def _new(x, dtype):
    """An uninitialised contiguous tensor of x's shape."""
    if dtype is x.dtype and x.is_contiguous():
        return _empty_like(x)
    return _empty(x.shape, dtype=dtype, device=x.device)


def unaligned(*tensors):
    """Whether one of the tensors (or Nones) does not start at a 16-byte boundary."""
    return any(t is not None and t.data_ptr() & 15 for t in tensors)


def aligned(t):
    """t, or a contiguous copy of it where it does not start at a 16-byte boundary."""
    return t.clone(memory_format=torch.contiguous_format) if unaligned(t) else t


def _room(t):
    """t, or an uninitialised tensor to fill in its place where it does not start at a 16-byte boundary."""
    return _empty(t.shape, dtype=t.dtype, device=t.device) if unaligned(t) else t


def put_back(*pairs):
    """Copy each (tensor, what was filled in its place) back."""
    for t, filled in pairs:
        if filled is not t:
            t.copy_(filled)


def _at(t):
    return None if t is None else t.data_ptr()


def _need(ok, message):
    if not ok:
        raise ValueError(message)


def _wrong(name, t, dtype, shape, device, contiguous=""):
    raise ValueError(f"{name}: expected {contiguous}{dtype} {list(shape)} on {device}, "
                     f"got {t.dtype} {list(t.shape)} (strides {list(t.stride())}) on {t.device}")


def _rows(name, t, dtype, shape, device):
    """A [T, D] tensor whose rows are contiguous; its row stride."""
    if t.dtype is not dtype or t.shape != shape or t.device != device:
        _wrong(name, t, dtype, shape, device)
    row, col = t.stride()
    T, D = shape
    if col == 1 and row >= D:
        return row
    if T <= 1:
        if col == 1 or D <= 1 or T == 0:
            return D
    elif D <= 1 and row >= D:
        return row
    raise ValueError(f"{name}: rows have to be contiguous and apart (strides {row}, {col} for {D} columns)")


def _dense(name, t, dtype, shape, device):
    if t.dtype is not dtype or t.shape != shape or t.device != device or not t.is_contiguous():
        _wrong(name, t, dtype, shape, device, "contiguous ")


def _gate_shape(cfg, gate, T, D, device):
    shape = gate.shape
    n = len(shape)
    if gate.dtype not in _TYPE or gate.device != device or not gate.is_contiguous() or not 1 <= n <= 2:
        raise ValueError(f"gate: expected contiguous bfloat16 or float32 on {device}, got {gate.dtype} {list(shape)} on "
                         f"{gate.device}")
    cfg.gate_type = _TYPE[gate.dtype]
    if n == 1:
        if shape[0] == D:
            cfg.gate_mode = abi.MOE_GATE_CHANNEL
            return
    elif shape[1] == D and (T % shape[0] == 0 if shape[0] else T == 0):
        # no gate rows go with no tokens; a group count is at least one
        cfg.gate_mode, cfg.gate_rows = abi.MOE_GATE_GROUP, shape[0] or 1
        return
    elif shape[0] == T and shape[1] == 1:
        cfg.gate_mode = abi.MOE_GATE_TOKEN
        return
    raise ValueError(f"gate {list(shape)}: expected [{D}], [G, {D}] with G dividing {T}, or [{T}, 1]")


def _norm_config(x, branch, gate, post_weight, pre_weight, residual_scale, branch_scale, eps, weight_offset):
    """The checked configuration shared by block_norm and its backward."""
    xt, shape, dev = x.dtype, x.shape, x.device
    if len(shape) != 2 or xt not in _TYPE or dev.type != "cuda":
        raise ValueError("x: expected a CUDA bfloat16 or float32 [T, D] tensor")
    T, D = shape
    if T >= _MOST or D >= _MOST:
        raise ValueError("x: sizes have to be below 2^31")
    kind = _FP32
    if pre_weight is not None:
        kind = pre_weight.dtype
        if kind not in _TYPE:
            raise ValueError("weights are bfloat16 or float32")
        _dense("pre_weight", pre_weight, kind, (D,), dev)
    if branch is None:
        if gate is not None or post_weight is not None:
            raise ValueError("a gate or post_weight needs a branch")
        branch_row = 0
    else:
        branch_row = _rows("branch", branch, _BF16, shape, dev)
        if post_weight is not None:
            if pre_weight is None:
                kind = post_weight.dtype
                if kind not in _TYPE:
                    raise ValueError("weights are bfloat16 or float32")
            _dense("post_weight", post_weight, kind, (D,), dev)
    cfg = _NormConfig(T, D, _TYPE[xt], _TYPE[kind], 0, 0, 0, residual_scale, branch_scale, eps, weight_offset,
                      _rows("x", x, xt, shape, dev), branch_row, 0, 0)
    if gate is not None:
        _gate_shape(cfg, gate, T, D, dev)
    return cfg


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
    ``y`` may be x and ``h`` may be branch (in place): for serving only, as the
    backward reads the x and branch that came in and would give wrong
    gradients from what replaced them.  ``stats``: a float32 [2, T] tensor for
    the backward to read (r of the branch with post_weight, r of y with
    pre_weight; the other row is left as it is)."""
    cfg = _norm_config(x, branch, gate, post_weight, pre_weight, residual_scale, branch_scale, eps, weight_offset)
    shape, dev = x.shape, x.device
    if y is not None:
        cfg.y_stride = _rows("y", y, x.dtype, shape, dev)
    if h is not None:
        _need(pre_weight is not None, "h needs a pre_weight")
        cfg.h_stride = _rows("h", h, _BF16, shape, dev)
    if stats is not None:
        _dense("stats", stats, _FP32, (2, shape[0]), dev)
    same = branch is None and y is None and residual_scale == 1.0
    _need(not same or pre_weight is not None, "nothing to compute: no branch, no pre_weight")

    def run(s):
        yy = y if y is not None or same else _new(x, x.dtype)
        hh = h if h is not None or pre_weight is None else _new(x, _BF16)
        status = _LIB.moe_block_norm_forward(_byref(cfg), x.data_ptr(), _at(branch), _at(gate), _at(post_weight),
                                             _at(pre_weight), _at(yy), _at(hh), _at(stats), s)
        if status:
            if status == _INVALID and unaligned(x, branch, gate, post_weight, pre_weight, y, h, stats):
                return _block_norm_realigned(cfg, x, branch, gate, post_weight, pre_weight, y, h, stats, same)
            raise abi.MoEError("moe_block_norm_forward", status)
        return (x if same else yy), hh

    return on_stream(run, dev, stream)


def _block_norm_realigned(cfg, x, branch, gate, post_weight, pre_weight, y, h, stats, same):
    """block_norm on aligned copies, on the current stream."""
    filled = _room(y), _room(h), aligned(stats)
    yy, hh = block_norm(aligned(x), aligned(branch), gate=aligned(gate), post_weight=aligned(post_weight),
                        pre_weight=aligned(pre_weight), residual_scale=cfg.residual_scale, branch_scale=cfg.branch_scale,
                        eps=cfg.eps, weight_offset=cfg.weight_offset, y=filled[0], h=filled[1], stats=filled[2])
    put_back((y, filled[0]), (h, filled[1]), (stats, filled[2]))
    return x if same else yy if y is None else y, hh if h is None else h


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
    forward's inputs (not overwritten since, by a call in place or otherwise)
    and ``stats``.  dx has x's type, dbranch is bfloat16,
    dgate has the gate's shape and type, the weights' gradients are float32."""
    cfg = _norm_config(x, branch, gate, post_weight, pre_weight, residual_scale, branch_scale, 1.0, weight_offset)
    shape, dev = x.shape, x.device
    T, D = shape
    _need((dh is not None) == (pre_weight is not None), "dh goes with pre_weight")
    _need(dy is not None or dh is not None, "no gradient given")
    if dy is not None:
        cfg.y_stride = _rows("dy", dy, x.dtype, shape, dev)
    if dh is not None:
        cfg.h_stride = _rows("dh", dh, _BF16, shape, dev)
    if post_weight is not None or pre_weight is not None:
        _need(stats is not None, "the norms' backward needs the forward's stats")
        _dense("stats", stats, _FP32, (2, T), dev)

    def run(s):
        dx = _new(x, x.dtype)
        dbranch = None if branch is None else _new(branch, _BF16)
        dgate = None if gate is None else _empty_like(gate)
        dpost = None if post_weight is None else _empty(D, dtype=_FP32, device=dev)
        dpre = None if pre_weight is None else _empty(D, dtype=_FP32, device=dev)
        ref = _byref(cfg)
        nb = _LIB.moe_block_norm_workspace_bytes(ref)
        ws = _empty(nb, dtype=torch.uint8, device=dev)
        status = _LIB.moe_block_norm_backward(ref, x.data_ptr(), _at(branch), _at(gate), _at(post_weight),
                                              _at(pre_weight), _at(stats), _at(dy), _at(dh), dx.data_ptr(), _at(dbranch),
                                              _at(dgate), _at(dpost), _at(dpre), ws.data_ptr(), nb, s)
        if status:
            if status == _INVALID and unaligned(x, branch, stats, dy, dh, gate, post_weight, pre_weight):
                return block_norm_backward(aligned(x), aligned(branch), aligned(stats), aligned(dy), aligned(dh),
                                           gate=aligned(gate), post_weight=aligned(post_weight),
                                           pre_weight=aligned(pre_weight), residual_scale=cfg.residual_scale,
                                           branch_scale=cfg.branch_scale, weight_offset=cfg.weight_offset)
            raise abi.MoEError("moe_block_norm_backward", status)
        return BlockNormGrads(dx, dbranch, dgate, dpost, dpre)

    return on_stream(run, dev, stream)


def _gate_config(logits, top_k, score, renormalize, scale):
    kind, shape, dev = logits.dtype, logits.shape, logits.device
    if len(shape) != 2 or kind not in _TYPE or dev.type != "cuda":
        raise ValueError("logits: expected a CUDA bfloat16 or float32 [T, E] tensor")
    if score not in _SCORE:
        raise ValueError("score: softmax or sigmoid")
    if shape[0] >= _MOST or shape[1] >= _MOST:
        raise ValueError("logits: sizes have to be below 2^31")
    return _GateConfig(shape[0], shape[1], top_k, _TYPE[kind], _SCORE[score], 1 if renormalize else 0, scale,
                       _rows("logits", logits, kind, shape, dev))


def _gate_options(cfg):
    return {"score": "sigmoid" if cfg.score == abi.MOE_SCORE_SIGMOID else "softmax", "renormalize": bool(cfg.renormalize),
            "scale": cfg.scale}


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
        _dense("select_bias", select_bias, _FP32, (logits.shape[1],), dev)
    if ids is not None:
        _dense("ids", ids, _INT32, shape, dev)
    if scores is not None:
        _dense("scores", scores, _FP32, shape, dev)

    def run(stream):
        i = _empty(shape, dtype=_INT32, device=dev) if ids is None else ids
        s = _empty(shape, dtype=_FP32, device=dev) if scores is None else scores
        status = _LIB.moe_topk_gate_forward(_byref(cfg), logits.data_ptr(), _at(select_bias), i.data_ptr(), s.data_ptr(),
                                            stream)
        if status:
            if status == _INVALID and unaligned(logits, select_bias, i, s):
                filled = _room(i), _room(s)
                topk_gate(aligned(logits), shape[1], **_gate_options(cfg), select_bias=aligned(select_bias), ids=filled[0],
                          scores=filled[1])
                put_back((i, filled[0]), (s, filled[1]))
                return i, s
            raise abi.MoEError("moe_topk_gate_forward", status)
        return i, s

    return on_stream(run, dev, stream)


def topk_gate_backward(logits, ids, d_scores, *, score="softmax", renormalize=False, scale=1.0, d_logits=None,
                       stream=None):
    """The gradient [T, E] of the logits (their type) from d_scores [T, top_k]
    (float32, MoELayer.backward's) at topk_gate's ids."""
    _need(ids.dim() == 2, "ids: expected [T, top_k]")
    cfg = _gate_config(logits, ids.shape[1], score, renormalize, scale)
    dev, shape = logits.device, (logits.shape[0], ids.shape[1])
    _dense("ids", ids, _INT32, shape, dev)
    _dense("d_scores", d_scores, _FP32, shape, dev)
    if d_logits is not None:
        _dense("d_logits", d_logits, logits.dtype, logits.shape, dev)

    def run(stream):
        d = _new(logits, logits.dtype) if d_logits is None else d_logits
        status = _LIB.moe_topk_gate_backward(_byref(cfg), logits.data_ptr(), ids.data_ptr(), d_scores.data_ptr(),
                                             d.data_ptr(), stream)
        if status:
            if status == _INVALID and unaligned(logits, ids, d_scores, d):
                filled = _room(d)
                topk_gate_backward(aligned(logits), aligned(ids), aligned(d_scores), **_gate_options(cfg), d_logits=filled)
                put_back((d, filled))
                return d
            raise abi.MoEError("moe_topk_gate_backward", status)
        return d

    return on_stream(run, dev, stream)


def _check_rng(p, rng, site, device):
    if not 0.0 <= p <= 1.0:
        raise ValueError(f"dropout: expected a probability, got {p}")
    if not 0 <= site < 1 << 32:
        raise ValueError("site: expected an integer of 32 bits")
    if rng is None:
        _need(p == 0.0, "dropout needs rng, an int64 tensor [seed, step] on the device")
    else:
        _dense("rng", rng, _INT64, (2,), device)


def dropout(x, p, rng, *, site=0, residual=None, out=None, stream=None):
    """keep * x / (1 - p) (+ residual) of a [T, D] bfloat16 or float32 tensor,
    x's type.  The mask is a function of rng (an int64 [2] tensor on x's
    device: seed and step), ``site`` (which call of a step this is) and the
    element's place in [T, D] alone; it is not stored, and ``dropout_backward``
    (or the same call on the gradient) draws it again.  rng is read on the
    device: a program, also within a captured graph, advances its step in place
    (``rng[1] += 1``) for new masks.  p counts in steps of 2^-16.  Dropped
    elements give 0 whatever x holds there.  ``out`` may be x or residual."""
    kind, shape, dev = x.dtype, x.shape, x.device
    if len(shape) != 2 or kind not in _TYPE or dev.type != "cuda":
        raise ValueError("x: expected a CUDA bfloat16 or float32 [T, D] tensor")
    if shape[0] >= _MOST or shape[1] >= _MOST:
        raise ValueError("x: sizes have to be below 2^31")
    _check_rng(p, rng, site, dev)
    cfg = _DropoutConfig(shape[0], shape[1], _TYPE[kind], site, p, _rows("x", x, kind, shape, dev))
    if residual is not None:
        cfg.residual_stride = _rows("residual", residual, kind, shape, dev)
    if out is not None:
        cfg.out_stride = _rows("out", out, kind, shape, dev)

    def run(s):
        o = _new(x, kind) if out is None else out
        status = _LIB.moe_dropout(_byref(cfg), x.data_ptr(), _at(residual), _at(rng), o.data_ptr(), s)
        if status:
            if status == _INVALID and unaligned(x, residual, rng, out):
                filled = _room(o)
                dropout(aligned(x), p, aligned(rng), site=site, residual=aligned(residual), out=filled)
                put_back((o, filled))
                return o
            raise abi.MoEError("moe_dropout", status)
        return o

    return on_stream(run, dev, stream)


def dropout_backward(dout, p, rng, *, site=0, dx=None, stream=None):
    """The gradient of dropout's x from that of its result, at the forward's
    p, rng and site (a residual's gradient is dout itself)."""
    return dropout(dout, p, rng, site=site, out=dx, stream=stream)


def _layer_norm_config(name, x, weight, bias, residual_scale, branch_scale, dropout, rng, site, eps):
    kind, shape, dev = x.dtype, x.shape, x.device
    if len(shape) != 2 or kind not in _TYPE or dev.type != "cuda":
        raise ValueError(f"{name}: expected a CUDA bfloat16 or float32 [T, D] tensor")
    T, D = shape
    if T >= _MOST or D >= _MOST:
        raise ValueError(f"{name}: sizes have to be below 2^31")
    par = _FP32
    if weight is not None or bias is not None:
        par = (bias if weight is None else weight).dtype
        if par not in _TYPE:
            raise ValueError("weight and bias are bfloat16 or float32")
        if weight is not None:
            _dense("weight", weight, par, (D,), dev)
        if bias is not None:
            _dense("bias", bias, par, (D,), dev)
    if dropout or rng is not None or site:
        _check_rng(dropout, rng, site, dev)
    return _LayerNormConfig(T, D, _TYPE[kind], _TYPE[par], residual_scale, branch_scale, eps, site, dropout,
                            _rows(name, x, kind, shape, dev))


_norm_bytes = {}


def _layer_norm_workspace(cfg, dev):
    """moe_layer_norm_workspace_bytes, remembered by what it depends on (0, of a
    configuration that the library refuses for whatever reason, is not)."""
    key = cfg.tokens, cfg.d_model, dev.index
    nb = _norm_bytes.get(key)
    if nb is None:
        nb = _LIB.moe_layer_norm_workspace_bytes(_byref(cfg))
        if nb:
            if len(_norm_bytes) >= 1024:
                _norm_bytes.clear()
            _norm_bytes[key] = nb
    return _empty(nb, dtype=torch.uint8, device=dev)


def layer_norm(x, branch=None, *, weight=None, bias=None, residual_scale=1.0, branch_scale=1.0, dropout=0.0, rng=None,
               site=0, eps=1e-5, y=None, h=None, stats=None, stream=None):
    """(y, h) of one block boundary:

        y = residual_scale * x + branch_scale * dropout(branch)
        h = (y - mean(y)) / sqrt(var(y) + eps) * weight + bias

    x: [T, D] bfloat16 or float32; branch: [T, D] bfloat16 or None (a norm
    alone: y is then x, and is written only where a ``y`` is given or the
    residual is scaled).  h is bfloat16.  weight, bias: [D] of one type, or
    None.  dropout, rng and site as in ``dropout``, whose mask on the branch
    this is.  ``y`` may be x and ``h`` may be branch (in place; the backward
    reads y alone).  ``stats``: a float32 [2, T] tensor for the backward to
    read (mean and 1 / sqrt(var + eps))."""
    cfg = _layer_norm_config("x", x, weight, bias, residual_scale, branch_scale, dropout, rng, site, eps)
    shape, dev = x.shape, x.device
    if branch is not None:
        cfg.branch_stride = _rows("branch", branch, _BF16, shape, dev)
    else:
        _need(dropout == 0.0, "dropout needs a branch")
    if y is not None:
        cfg.y_stride = _rows("y", y, x.dtype, shape, dev)
    if h is not None:
        cfg.h_stride = _rows("h", h, _BF16, shape, dev)
    if stats is not None:
        _dense("stats", stats, _FP32, (2, shape[0]), dev)
    same = branch is None and y is None and residual_scale == 1.0

    def run(s):
        yy = y if y is not None or same else _new(x, x.dtype)
        hh = h if h is not None else _new(x, _BF16)
        status = _LIB.moe_layer_norm_forward(_byref(cfg), x.data_ptr(), _at(branch), _at(weight), _at(bias), _at(rng),
                                             _at(yy), hh.data_ptr(), _at(stats), s)
        if status:
            if status == _INVALID and unaligned(x, branch, weight, bias, rng, y, h, stats):
                filled = _room(y), _room(h), aligned(stats)
                yy, hh = layer_norm(aligned(x), aligned(branch), weight=aligned(weight), bias=aligned(bias),
                                    residual_scale=cfg.residual_scale, branch_scale=cfg.branch_scale, dropout=dropout,
                                    rng=aligned(rng), site=site, eps=cfg.eps, y=filled[0], h=filled[1], stats=filled[2])
                put_back((y, filled[0]), (h, filled[1]), (stats, filled[2]))
                return x if same else yy if y is None else y, hh if h is None else h
            raise abi.MoEError("moe_layer_norm_forward", status)
        return (x if same else yy), hh

    return on_stream(run, dev, stream)


class LayerNormGrads(NamedTuple):
    dx: torch.Tensor
    dbranch: Optional[torch.Tensor]
    dweight: Optional[torch.Tensor]
    dbias: Optional[torch.Tensor]


def layer_norm_backward(y, stats, dh, dy=None, *, weight=None, bias=None, branch=True, residual_scale=1.0,
                        branch_scale=1.0, dropout=0.0, rng=None, site=0, stream=None):
    """Gradients (LayerNormGrads) of layer_norm's inputs from ``dh`` (bfloat16)
    and ``dy`` (y's type; None: zero), with the forward's y and ``stats``.
    branch: whether the forward had one (dbranch is bfloat16).  weight and
    bias: the forward's; each that is given gets its gradient, float32.  dropout,
    rng and site: the forward's."""
    cfg = _layer_norm_config("y", y, weight, bias, residual_scale, branch_scale, dropout, rng, site, 1.0)
    shape, dev = y.shape, y.device
    T, D = shape
    cfg.h_stride = _rows("dh", dh, _BF16, shape, dev)
    if dy is not None:
        cfg.y_stride = _rows("dy", dy, y.dtype, shape, dev)
    _dense("stats", stats, _FP32, (2, T), dev)
    _need(branch or dropout == 0.0, "dropout needs a branch")

    def run(s):
        dx = _new(y, y.dtype)
        dbranch = _new(y, _BF16) if branch else None
        dweight = None if weight is None else _empty(D, dtype=_FP32, device=dev)
        dbias = None if bias is None else _empty(D, dtype=_FP32, device=dev)
        ws = _layer_norm_workspace(cfg, dev)
        status = _LIB.moe_layer_norm_backward(_byref(cfg), y.data_ptr(), _at(weight), stats.data_ptr(), _at(rng), _at(dy),
                                              dh.data_ptr(), dx.data_ptr(), _at(dbranch), _at(dweight), _at(dbias),
                                              ws.data_ptr(), ws.numel(), s)
        if status:
            if status == _INVALID and unaligned(y, stats, dh, dy, weight, rng):
                return layer_norm_backward(aligned(y), aligned(stats), aligned(dh), aligned(dy), weight=aligned(weight),
                                           bias=bias, branch=branch, residual_scale=cfg.residual_scale,
                                           branch_scale=cfg.branch_scale, dropout=dropout, rng=aligned(rng), site=site)
            raise abi.MoEError("moe_layer_norm_backward", status)
        return LayerNormGrads(dx, dbranch, dweight, dbias)

    return on_stream(run, dev, stream)
