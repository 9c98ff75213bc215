"""Orthogonalised updates (Muon) of stacked expert weights, on torch tensors.

``orthogonalize`` gives the Newton-Schulz polynomial of a stack of matrices,
``muon_update`` is a whole optimiser step in place, and ``Muon`` keeps the
momenta and the workspace of a set of weights.  The computation runs in the
CUDA library (``moe_orthogonalize``, ``moe_muon_update`` of the C ABI).

Weights are stacks [E, rows, cols], such as W2 [E, D, F].  W13 [E, 2F, D]
holds two matrices an expert: its view [2E, F, D] updates gate and up apart.
Tensors that do not start at a 16-byte boundary (views into a flat buffer) are
worked on in aligned copies, as in ``block``.
"""

import math

import torch

from . import abi
from .block import _TYPE, _dense, _need, aligned, on_stream, put_back, unaligned

# a s + b s^3 + c s^5: a steep start for small singular values; five steps take [1e-3, 1] near 1
COEFFICIENTS = (3.4445, -4.7750, 2.0315)

# bytes a workspace that a call makes for itself may take, unless one matrix needs more
WORKSPACE_LIMIT = 4 << 30

_error_words = {}


def _config(shape, steps, coefficients, eps):
    _need(len(shape) == 3, "expected a stack of matrices [E, rows, cols]")
    _need(max(shape) < 1 << 31, "sizes have to be below 2^31")
    _need(1 <= steps <= abi.MOE_MUON_MAX_STEPS, "steps: 1 to 16")
    cfg = abi.moe_muon_config(shape[0], shape[1], shape[2], steps)
    cfg.eps = eps
    table = coefficients if len(coefficients) and hasattr(coefficients[0], "__len__") else [coefficients] * steps
    _need(len(table) == steps and all(len(t) == 3 for t in table),
          "coefficients: (a, b, c), or one triple for each step")
    for s, triple in enumerate(table):
        cfg.coefficients[s][:] = triple
    return cfg


def _error_word(device):
    """The address of the library's error word on `device`, which is current."""
    word = _error_words.get(device)
    if word is None:
        word = _error_words[device] = abi.moe_muon_error_word()
    return word


def error_bits(device="cuda"):
    """The MOE_DEV_ERR_* bits that updates on `device` have set (0: none); synchronises and clears them."""
    with torch.cuda.device(torch.device(device)):
        return abi.moe_muon_get_error()


def workspace(E, rows, cols, *, matrices=None, device="cuda"):
    """A workspace for stacks of E matrices [rows, cols], worked through in
    runs of `matrices` (default: as many as 4 GiB hold)."""
    cfg = _config((E, rows, cols), 1, COEFFICIENTS, 1.0)
    if matrices is None:
        one = abi.moe_muon_workspace_bytes(cfg, 2) - abi.moe_muon_workspace_bytes(cfg, 1)
        matrices = max(1, min(E, WORKSPACE_LIMIT // max(1, one)))
    return torch.empty(abi.moe_muon_workspace_bytes(cfg, matrices), dtype=torch.uint8, device=device)


def _workspace(given, shape, device):
    if given is None:
        return workspace(*shape, device=device)
    _need(given.dtype == torch.uint8 and given.is_contiguous() and given.device == device and given.data_ptr() % 256 == 0,
          "workspace: expected a contiguous uint8 tensor on the weights' device that starts at a 256-byte boundary")
    return given


def orthogonalize(x, *, steps=5, coefficients=COEFFICIENTS, eps=1e-7, out=None, workspace=None, stream=None):
    """The orthogonalised x [E, rows, cols] (bfloat16 or float32), bfloat16:
    `steps` of X <- a X + (b A + c A A) X, A = X X^T, from x / (|x| + eps)."""
    _need(x.is_cuda and x.dtype in _TYPE and x.is_contiguous(), "x: expected a contiguous CUDA bfloat16 or float32 stack")
    cfg = _config(tuple(x.shape), steps, coefficients, eps)
    dev = x.device
    if out is not None:
        _dense("out", out, torch.bfloat16, tuple(x.shape), dev)

    def run(s):
        o = torch.empty(x.shape, dtype=torch.bfloat16, device=dev) if out is None else out
        ws = _workspace(workspace, x.shape, dev)

        def call(u, filled):
            abi.moe_orthogonalize(cfg, u, _TYPE[x.dtype], filled, ws, ws.numel(), _error_word(dev), s)

        try:
            call(x, o)
        except abi.MoEError:
            if not unaligned(x, o):
                raise
            filled = aligned(o)
            call(aligned(x), filled)
            put_back((o, filled))
        return o

    return on_stream(run, dev, stream)


def muon_update(weight, grad, momentum, *, lr, mu=0.95, nesterov=True, weight_decay=0.0, scale=None, steps=5,
                coefficients=COEFFICIENTS, eps=1e-7, weight_bf16=None, workspace=None, stream=None):
    """One step in place on `weight` (bfloat16 or float32 [E, rows, cols]) and
    `momentum` (float32):

        momentum = mu * momentum + grad
        weight = (1 - lr * weight_decay) * weight
                 - lr * scale * orthogonalize(grad + mu * momentum)

    (without nesterov: of the momentum).  scale: default 0.2 sqrt(max(rows,
    cols)), which gives updates the RMS of an Adam step.  weight_bf16: a
    bfloat16 copy of a float32 weight to refresh, as the layer reads it.
    Where a device wait runs out of time (error_bits), weights whose products
    were not finished stay as they were; the momentum has taken its step."""
    _need(weight.is_cuda and weight.dtype in _TYPE and weight.is_contiguous(),
          "weight: expected a contiguous CUDA bfloat16 or float32 stack")
    _need(grad.dtype in _TYPE, "grad: bfloat16 or float32")
    shape, dev = tuple(weight.shape), weight.device
    cfg = _config(shape, steps, coefficients, eps)
    _dense("grad", grad, grad.dtype, shape, dev)
    _dense("momentum", momentum, torch.float32, shape, dev)
    if weight_bf16 is not None:
        _need(weight.dtype == torch.float32, "weight_bf16 is the copy of a float32 weight")
        _dense("weight_bf16", weight_bf16, torch.bfloat16, shape, dev)
    if scale is None:
        scale = 0.2 * math.sqrt(max(shape[1], shape[2]))
    rates = abi.moe_muon_rates(lr, mu, weight_decay, scale, 1 if nesterov else 0)

    def run(s):
        ws = _workspace(workspace, shape, dev)

        def call(w, g, m, copy):
            abi.moe_muon_update(cfg, rates, w, _TYPE[weight.dtype], g, _TYPE[grad.dtype], m, copy, ws, ws.numel(),
                                _error_word(dev), s)

        try:
            call(weight, grad, momentum, weight_bf16)
        except abi.MoEError:
            if not unaligned(weight, grad, momentum, weight_bf16):
                raise
            filled = aligned(weight), aligned(momentum), aligned(weight_bf16)
            call(filled[0], aligned(grad), *filled[1:])
            put_back((weight, filled[0]), (momentum, filled[1]), (weight_bf16, filled[2]))

    on_stream(run, dev, stream)


class Muon:
    """The optimiser of a list of stacked weights: FP32 momenta (and, with
    master=True, FP32 master copies of bfloat16 weights) and one workspace
    that every step shares, so steps of one object run on one stream.  A step
    only enqueues: error_bits() tells, whenever the program asks, whether a
    device wait ran out of time and left weights without their update."""

    def __init__(self, weights, *, lr, mu=0.95, nesterov=True, weight_decay=0.0, steps=5, coefficients=COEFFICIENTS,
                 eps=1e-7, master=False):
        self.weights = list(weights)
        self.lr, self.weight_decay = lr, weight_decay
        self.options = dict(mu=mu, nesterov=nesterov, steps=steps, coefficients=coefficients, eps=eps)
        self.momenta = [torch.zeros(w.shape, dtype=torch.float32, device=w.device) for w in self.weights]
        self.masters = [w.float() if master and w.dtype == torch.bfloat16 else None for w in self.weights]
        sizes = [workspace(*w.shape, device="meta").numel() for w in self.weights]
        self.workspace = torch.empty(max(sizes, default=0), dtype=torch.uint8,
                                     device=self.weights[0].device if self.weights else "cuda")

    def step(self, grads, stream=None):
        _need(len(grads) == len(self.weights), "one gradient for each weight")
        for w, g, m, f in zip(self.weights, grads, self.momenta, self.masters):
            muon_update(w if f is None else f, g, m, lr=self.lr, weight_decay=self.weight_decay,
                        weight_bf16=None if f is None else w, workspace=self.workspace, stream=stream, **self.options)
