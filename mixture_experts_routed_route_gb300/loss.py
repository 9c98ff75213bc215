"""The loss that closes a training step, on torch tensors: softmax cross entropy
on top of the output projection (``linear_cross_entropy``) and its backward.

The logits [T, V] are never in memory as a whole: the forward keeps a maximum
and a sum a token and tile, the backward forms a piece of the vocabulary at a
time.  The computation runs in the CUDA library (``moe_linear_ce_*`` of the C
ABI).  Streams, devices and tensors that do not start at a 16-byte boundary are
treated as in ``block``; a device wait that ran out of time shows in
``optim.error_bits``, the word that the library keeps for each device.
"""

import torch

from . import abi
from .block import _BF16, _FP32, _INT32, _INT64, _at, _dense, _empty, _MOST, _need, _room, _rows, aligned, on_stream
from .block import put_back, unaligned
from .optim import _error_word

# bytes that a backward call's own workspace may take for a piece's gradient of the logits, unless 256 entries need more
PIECE_BYTES = 512 << 20

_TARGET = {_INT32: 4, _INT64: 8}


def _config(h, weight, targets, ignore_index, logit_scale, z_weight):
    if len(h.shape) != 2 or h.dtype is not _BF16 or h.device.type != "cuda":
        raise ValueError("h: expected a CUDA bfloat16 [T, D] tensor")
    T, D = h.shape
    if len(weight.shape) != 2 or weight.shape[0] < 1:
        raise ValueError("weight: expected [V, D]")
    V = weight.shape[0]
    if T >= _MOST or D >= _MOST or V >= _MOST:
        raise ValueError("sizes have to be below 2^31")
    _dense("weight", weight, _BF16, (V, D), h.device)
    if targets.dtype not in _TARGET:
        raise ValueError("targets: expected int32 or int64")
    _dense("targets", targets, targets.dtype, (T,), h.device)
    if not -(1 << 63) <= ignore_index < 1 << 63:
        raise ValueError("ignore_index: expected an integer of 64 bits")
    return abi.moe_linear_ce_config(T, D, V, _TARGET[targets.dtype], logit_scale, z_weight, ignore_index,
                                    _rows("h", h, _BF16, h.shape, h.device))


def _workspace_bytes(cfg, backward, piece):
    if piece is None:
        rows = -(-cfg.tokens // 256) * 256
        piece = max(256, PIECE_BYTES // (2 * max(1, rows)))
    _need(1 <= piece < _MOST, "piece: expected a number of vocabulary entries")
    return abi.moe_linear_ce_workspace_bytes(cfg, backward, piece)


def workspace(T, D, V, *, backward=True, piece=None, device="cuda"):
    """A workspace for calls on up to T tokens: of the forward or the backward,
    which works in pieces of `piece` vocabulary entries (default: as many as
    512 MiB hold; a larger workspace means larger pieces)."""
    _need(0 <= T < _MOST and 0 < D < _MOST and 0 < V < _MOST, "sizes: expected T >= 0, D and V >= 1, all below 2^31")
    cfg = abi.moe_linear_ce_config(T, D, V, 8, 1.0, 0.0, -100, 0)
    device = torch.device(device)
    with torch.cuda.device(device):
        return _empty(_workspace_bytes(cfg, backward, piece), dtype=torch.uint8, device=device)


def _workspace(given, cfg, backward, device):
    if given is None:
        return _empty(_workspace_bytes(cfg, backward, None), dtype=torch.uint8, device=device)
    _need(given.dtype == torch.uint8 and given.is_contiguous() and given.device == device and given.data_ptr() % 256 == 0,
          "workspace: expected a contiguous uint8 tensor on h's device that starts at a 256-byte boundary")
    return given


def linear_cross_entropy(h, weight, targets, *, ignore_index=-100, logit_scale=1.0, z_weight=0.0, loss=None, lse=None,
                         workspace=None, stream=None):
    """(loss, lse), float32 [T], of logits = logit_scale * h @ weight.T:

        lse = log(sum(exp(logits)));  loss = lse - logits[target] + z_weight * lse^2

    h: [T, D] bfloat16; weight: [V, D] bfloat16; targets: [T] int32 or int64.
    Where the target is ignore_index both are 0 and h may hold anything; any
    other target outside [0, V) gives a NaN loss.  D is a multiple of 8."""
    cfg = _config(h, weight, targets, ignore_index, logit_scale, z_weight)
    dev, T = h.device, h.shape[0]
    if loss is not None:
        _dense("loss", loss, _FP32, (T,), dev)
    if lse is not None:
        _dense("lse", lse, _FP32, (T,), dev)

    def run(s):
        value = _empty(T, dtype=_FP32, device=dev) if loss is None else loss
        total = _empty(T, dtype=_FP32, device=dev) if lse is None else lse
        ws = _workspace(workspace, cfg, False, dev)
        status = abi.LIB.moe_linear_ce_forward(cfg, h.data_ptr(), weight.data_ptr(), targets.data_ptr(), value.data_ptr(),
                                               total.data_ptr(), ws.data_ptr(), ws.numel(), _error_word(dev), s)
        if status:
            if status == abi.MOE_ERR_INVALID_ARG and unaligned(h, weight, targets, value, total):
                filled = _room(value), _room(total)
                linear_cross_entropy(aligned(h), aligned(weight), aligned(targets), ignore_index=ignore_index,
                                     logit_scale=cfg.logit_scale, z_weight=cfg.z_weight, loss=filled[0], lse=filled[1],
                                     workspace=workspace)
                put_back((value, filled[0]), (total, filled[1]))
                return value, total
            raise abi.MoEError("moe_linear_ce_forward", status)
        return value, total

    return on_stream(run, dev, stream)


def linear_cross_entropy_backward(h, weight, targets, lse, d_loss, *, ignore_index=-100, logit_scale=1.0, z_weight=0.0,
                                  need_dh=True, need_dweight=True, dh=None, dweight=None, workspace=None, stream=None):
    """(dh [T, D], dweight [V, D]), bfloat16, from d_loss (float32 [T], the
    gradient of each token's loss: 1 / tokens for a mean) and the forward's
    inputs and lse; None in the place of a gradient that is not needed.  Rows
    that do not count get zeros in dh."""
    cfg = _config(h, weight, targets, ignore_index, logit_scale, z_weight)
    dev, T = h.device, h.shape[0]
    _dense("lse", lse, _FP32, (T,), dev)
    _dense("d_loss", d_loss, _FP32, (T,), dev)
    _need(need_dh or need_dweight, "no gradient asked for")
    if dh is not None:
        _need(need_dh, "dh is not needed")
        _dense("dh", dh, _BF16, h.shape, dev)
    if dweight is not None:
        _need(need_dweight, "dweight is not needed")
        _dense("dweight", dweight, _BF16, weight.shape, dev)

    def run(s):
        gh = _empty(h.shape, dtype=_BF16, device=dev) if dh is None and need_dh else dh
        gw = _empty(weight.shape, dtype=_BF16, device=dev) if dweight is None and need_dweight else dweight
        ws = _workspace(workspace, cfg, True, dev)
        status = abi.LIB.moe_linear_ce_backward(cfg, h.data_ptr(), weight.data_ptr(), targets.data_ptr(), lse.data_ptr(),
                                                d_loss.data_ptr(), _at(gh), _at(gw), ws.data_ptr(), ws.numel(),
                                                _error_word(dev), s)
        if status:
            if status == abi.MOE_ERR_INVALID_ARG and unaligned(h, weight, targets, lse, d_loss, gh, gw):
                filled = _room(gh) if need_dh else None, _room(gw) if need_dweight else None
                linear_cross_entropy_backward(aligned(h), aligned(weight), aligned(targets), aligned(lse), aligned(d_loss),
                                              ignore_index=ignore_index, logit_scale=cfg.logit_scale, z_weight=cfg.z_weight,
                                              need_dh=need_dh, need_dweight=need_dweight, dh=filled[0], dweight=filled[1],
                                              workspace=workspace)
                put_back(*((t, f) for t, f in zip((gh, gw), filled) if t is not None))
                return gh, gw
            raise abi.MoEError("moe_linear_ce_backward", status)
        return gh, gw

    return on_stream(run, dev, stream)
