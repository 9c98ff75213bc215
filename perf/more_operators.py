"""Timed cases of what closes a training step around the routed experts, and their plain forms.

Three operators:

* ``dropout``: out = x * keep / (1 - p) (+ residual), the mask from a counter-based
  generator (Philox4x32 with ten rounds; element e of the flat tensor takes 16 of the
  128 bits of counter (e / 8, site, step) under the key ``seed``) and never stored;
* ``layer_norm``: the residual of a block with dropout on its branch and the norm
  before the next one in one pass,
      y = residual_scale * x + branch_scale * dropout(branch)
      h = (y - mean(y)) / sqrt(var(y) + eps) * weight + bias
  and its backward pass (gradients of x, branch, weight and bias);
* ``cross_entropy``: the softmax cross entropy of logits = h @ weight^T over a
  large vocabulary, whose logits are not kept,
      loss = lse - logit[target] + z_weight * lse^2,   lse = log(sum exp(logits))
  with ignored targets, and the gradients of h and weight.

``run`` computes a case in its plain form (elementary torch operations in 32
bits, rounded once at the end) or, with ``own``, through the framework.
Widths are those of the framework's workloads (256, 1408, 2048, 7168) and odd
ones; vocabularies are powers of two and odd sizes.
"""

import math

import numpy as np
import torch

own = False

EPS = 1e-5
ALPHA, BETA = 0.95, 0.7
SITE = 5
IGNORE = -100

_TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
_BYTES = {"bf16": 2, "fp32": 4}


# -------------------------------------------------------------------- cases

def _dropout(name, T, D, dtype, p, residual):
    c = {"op": "dropout", "T": T, "D": D, "dtype": dtype, "p": p, "residual": residual}
    return dict(c, name=name) if name else c


def _norm(name, op, T, D, residual, branch, p, params="bf16"):
    c = {"op": op, "T": T, "D": D, "residual": residual, "branch": branch, "p": p, "params": params}
    return dict(c, name=name) if name else c


def _ce(name, op, T, D, V, ignored=0, z=0.0):
    c = {"op": op, "T": T, "D": D, "V": V, "ignored": ignored, "z": z}
    return dict(c, name=name) if name else c


def listed():
    return [
        # the smallest workload's experts' output: latency
        _dropout("dropout 128x256", 128, 256, "bf16", 0.1, False),
        # a long packed batch of the D=7168 model
        _dropout("dropout 16384x7168", 16384, 7168, "bf16", 0.1, False),
        # a width that no vector divides, added to an FP32 residual stream
        _dropout("dropout 4099x1411 residual", 4099, 1411, "fp32", 0.2, True),
        # one decode token between two blocks: latency, no dropout
        _norm("layer norm decode 1x7168", "layer_norm_forward", 1, 7168, "bf16", True, 0.0),
        # the E=384 training step's tokens, residual dropout
        _norm("layer norm forward 2048x7168", "layer_norm_forward", 2048, 7168, "bf16", True, 0.1),
        # its backward
        _norm("layer norm backward 2048x7168", "layer_norm_backward", 2048, 7168, "bf16", True, 0.1),
        # a ragged batch and a width that no vector divides, FP32 residual stream and parameters
        _norm("layer norm backward 1531x1411", "layer_norm_backward", 1531, 1411, "fp32", True, 0.0, "fp32"),
        # the log-likelihood of one token at decode: the vocabulary's weights are read once
        _ce("cross entropy forward 1x2048x131072", "cross_entropy_forward", 1, 2048, 131072),
        # the E=384 training step's tokens
        _ce("cross entropy forward 2048x7168x131072", "cross_entropy_forward", 2048, 7168, 131072, 0, 1e-4),
        # a small model's step: launches and short products count
        _ce("cross entropy backward 512x256x32768", "cross_entropy_backward", 512, 256, 32768),
        # a fine-tuning batch whose prompts take no loss, an odd vocabulary
        _ce("cross entropy backward 1531x1408x50021", "cross_entropy_backward", 1531, 1408, 50021, 459, 1e-4),
        # a training step's tokens of the D=2048 model
        _ce("cross entropy backward 4096x2048x131072", "cross_entropy_backward", 4096, 2048, 131072),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["dropout", "layer_norm_forward", "layer_norm_backward", "cross_entropy_forward",
                     "cross_entropy_backward"])
    if op.startswith("cross"):
        D = rng.choice([256, 1408, 2048, 7168, 8 * _log(rng, 8, 512)])
        V = rng.choice([32768, 131072, _log(rng, 1000, 131072), _log(rng, 1000, 131072) | 1])
        T = _log(rng, 1, max(1, min(8192, 4096 * 2048 * 131072 // (V * D))))
        ignored = rng.choice([0, T // 10, T // 2])
        return _ce(None, op, T, D, V, ignored, rng.choice([0.0, 1e-4]))
    D = rng.choice([256, 2048, 7168, _log(rng, 64, 8192), _log(rng, 64, 8192) | 1])
    T = _log(rng, 1, max(1, min(16384, 4096 * 7168 // D)))
    p = rng.choice([0.0, 0.1, 0.25, 0.5])
    if op == "dropout":
        return _dropout(None, T, D, rng.choice(["bf16", "fp32"]), p or 0.1, rng.random() < 0.5)
    return _norm(None, op, T, D, rng.choice(["bf16", "fp32"]), rng.random() < 0.8, p, rng.choice(["bf16", "fp32"]))


# ------------------------------------------------------------------- inputs

def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    rnd = lambda *shape: torch.randn(shape, generator=g, device=dev)  # noqa: E731
    s = {"case": case}
    op, T, D = case["op"], case["T"], case["D"]
    if op.startswith("cross"):
        V = case["V"]
        # an output projection, some words common; targets that the rows point to
        s["weight"] = torch.empty((V, D), dtype=torch.bfloat16, device=dev)
        for v in range(0, V, 16384):
            n = min(16384, V - v)
            s["weight"][v:v + n] = 2.0 * D ** -0.5 * rnd(n, D)
        s["targets"] = (torch.rand(T, generator=g, device=dev) ** 3 * V).long().clamp(max=V - 1)
        s["h"] = (rnd(T, D) + 2.5 * s["weight"][s["targets"]].float()).to(torch.bfloat16)
        s["targets"][torch.randperm(T, generator=g, device=dev)[:case["ignored"]]] = IGNORE
        if op == "cross_entropy_backward":
            # what the forward pass saved, and a mean over tokens of different weights
            s["lse"] = torch.zeros(T, device=dev)
            on = s["targets"] != IGNORE
            for t in range(0, T, 1024):
                s["lse"][t:t + 1024] = _lse(_logits(s, slice(t, t + 1024)))
            s["lse"] = torch.where(on, s["lse"], 0.0)
            s["d_loss"] = (0.5 + torch.rand(T, generator=g, device=dev)) / max(1, T - case["ignored"])
        return s
    # the generator's key and the step it is at, as a training loop keeps them on the device
    s["rng"] = torch.tensor([0x1234567 * (seed + 1), 17 + seed], dtype=torch.int64, device=dev)
    if op == "dropout":
        kind = _TYPES[case["dtype"]]
        s["x"] = rnd(T, D).to(kind)
        s["residual"] = (2.0 * rnd(T, D)).to(kind) if case["residual"] else None
        return s
    res, par = _TYPES[case["residual"]], _TYPES[case["params"]]
    # a residual stream grows over the layers, has a few large channels and a mean that is not zero
    channels = torch.where(torch.rand(D, generator=g, device=dev) < 0.01, 20.0, 1.0)
    x = 2.0 * channels * rnd(T, D) + 0.5
    s["weight"] = (1.0 + 0.1 * rnd(D)).to(par)
    s["bias"] = (0.1 * rnd(D)).to(par)
    if op == "layer_norm_forward":
        s["x"] = x.to(res)
        s["branch"] = (0.3 * rnd(T, D)).to(torch.bfloat16) if case["branch"] else None
    else:
        s["y"] = x.to(res)
        y = s["y"].float()
        mean = y.mean(1, keepdim=True)
        # what the forward pass saved
        s["stats"] = torch.stack((mean[:, 0], torch.rsqrt(((y - mean) ** 2).mean(1) + EPS)))
        s["dy"] = rnd(T, D).to(res)
        s["dh"] = rnd(T, D).to(torch.bfloat16)
    return s


# -------------------------------------------------------------- plain forms

def _mul32(a, b):
    """High and low words of a 32 x 32 bit product, a a tensor in int64, b a number."""
    low, high = a * (b & 0xFFFF), a * (b >> 16)
    return (high + (low >> 16)) >> 16, (((high & 0xFFFF) << 16) + low) & 0xFFFFFFFF


def _threshold(p):
    return int(math.floor(p * 65536 + 0.5))


def _kept(rng, n, p):
    """What each of n elements is multiplied by: 0 or 1 / (1 - p), p in steps of 2^-16."""
    seed, step = rng[0], rng[1] & 0xFFFFFFFF
    k0, k1 = seed & 0xFFFFFFFF, (seed >> 32) & 0xFFFFFFFF
    group = torch.arange((n + 7) // 8, dtype=torch.int64, device=rng.device)
    c0, c1 = group & 0xFFFFFFFF, group >> 32
    c2, c3 = torch.full_like(group, SITE), step.expand_as(group)
    for r in range(10):
        h0, l0 = _mul32(c0, 0xD2511F53)
        h1, l1 = _mul32(c2, 0xCD9E8D57)
        c0, c1, c2, c3 = h1 ^ c1 ^ ((k0 + r * 0x9E3779B9) & 0xFFFFFFFF), l1, h0 ^ c3 ^ ((k1 + r * 0xBB67AE85) & 0xFFFFFFFF), l0
    bits = torch.stack([w for c in (c0, c1, c2, c3) for w in (c & 0xFFFF, c >> 16)], 1).reshape(-1)[:n]
    t = _threshold(p)
    return torch.where(bits >= t, 65536.0 / (65536 - t), 0.0)


def _dropped(s, x):
    p = s["case"]["p"]
    if p == 0.0:
        return x
    keep = _kept(s["rng"], x.numel(), p).view(x.shape)
    return torch.where(keep > 0, x * keep, 0.0)


def _plain_dropout(s):
    x = _dropped(s, s["x"].float())
    if s["residual"] is not None:
        x = x + s["residual"].float()
    return x.to(s["x"].dtype)


def _norm_forward(s):
    y = ALPHA * s["x"].float()
    if s["branch"] is not None:
        y = y + BETA * _dropped(s, s["branch"].float())
    mean = y.mean(1, keepdim=True)
    r = torch.rsqrt(((y - mean) ** 2).mean(1, keepdim=True) + EPS)
    h = (y - mean) * r * s["weight"].float() + s["bias"].float()
    return {"y": y.to(s["x"].dtype), "h": h.to(torch.bfloat16), "stats": torch.cat((mean, r), 1).t()}


def _norm_backward(s):
    y, dy, dh = s["y"].float(), s["dy"].float(), s["dh"].float()
    mean, r = s["stats"][0][:, None], s["stats"][1][:, None]
    n = (y - mean) * r
    a = dh * s["weight"].float()
    d = dy + r * (a - a.mean(1, keepdim=True) - n * (a * n).mean(1, keepdim=True))
    out = {"dx": (ALPHA * d).to(s["y"].dtype), "dweight": (dh * n).sum(0), "dbias": dh.sum(0)}
    if s["case"]["branch"]:
        out["dbranch"] = (BETA * _dropped(s, d)).to(torch.bfloat16)
    return out


def _logits(s, rows=slice(None)):
    return torch.matmul(s["h"][rows].float(), s["weight"].float().t())


def _lse(logits):
    top = logits.max(1, keepdim=True).values
    return torch.log(torch.exp(logits - top).sum(1)) + top[:, 0]


def _ce_forward(s):
    logits = _logits(s)
    lse = _lse(logits)
    on = s["targets"] != IGNORE
    hit = logits.gather(1, s["targets"].clamp(min=0)[:, None])[:, 0]
    loss = lse - hit + s["case"]["z"] * lse * lse
    return {"loss": torch.where(on, loss, 0.0), "lse": torch.where(on, lse, 0.0)}


def _ce_backward(s):
    on = (s["targets"] != IGNORE).float()[:, None]
    logits = _logits(s)
    lse = s["lse"][:, None]
    g = torch.exp(logits - lse) * (1.0 + 2.0 * s["case"]["z"] * lse)
    g.scatter_add_(1, s["targets"].clamp(min=0)[:, None], torch.full_like(lse, -1.0))
    g = g * (s["d_loss"][:, None] * on)
    dh = torch.matmul(g, s["weight"].float())
    return {"dh": dh.to(torch.bfloat16), "dweight": torch.matmul(g.t(), s["h"].float()).to(torch.bfloat16)}


_PLAIN = {"dropout": _plain_dropout, "layer_norm_forward": _norm_forward, "layer_norm_backward": _norm_backward,
          "cross_entropy_forward": _ce_forward, "cross_entropy_backward": _ce_backward}


# ------------------------------------------------------------ the framework

def _framework(s):
    from mixture_experts_routed_route_gb300 import block, loss
    c = s["case"]
    op = c["op"]
    if op == "dropout":
        return block.dropout(s["x"], c["p"], s["rng"], site=SITE, residual=s["residual"])
    if op == "layer_norm_forward":
        stats = torch.empty((2, c["T"]), dtype=torch.float32, device=s["x"].device)
        y, h = block.layer_norm(s["x"], s["branch"], weight=s["weight"], bias=s["bias"], residual_scale=ALPHA,
                                branch_scale=BETA, dropout=c["p"] if c["branch"] else 0.0, rng=s["rng"], site=SITE,
                                eps=EPS, stats=stats)
        return {"y": y, "h": h, "stats": stats}
    if op == "layer_norm_backward":
        r = block.layer_norm_backward(s["y"], s["stats"], s["dh"], s["dy"], weight=s["weight"], bias=s["bias"],
                                      branch=c["branch"], residual_scale=ALPHA, branch_scale=BETA,
                                      dropout=c["p"] if c["branch"] else 0.0, rng=s["rng"], site=SITE)
        out = {"dx": r.dx, "dweight": r.dweight, "dbias": r.dbias}
        if c["branch"]:
            out["dbranch"] = r.dbranch
        return out
    if op == "cross_entropy_forward":
        value, lse = loss.linear_cross_entropy(s["h"], s["weight"], s["targets"], ignore_index=IGNORE, z_weight=c["z"])
        return {"loss": value, "lse": lse}
    dh, dweight = loss.linear_cross_entropy_backward(s["h"], s["weight"], s["targets"], s["lse"], s["d_loss"],
                                                     ignore_index=IGNORE, z_weight=c["z"])
    return {"dh": dh, "dweight": dweight}


def run(state):
    return _framework(state) if own else _PLAIN[state["case"]["op"]](state)


# --------------------------------------------------------------------- work

def work(case):
    op, T, D = case["op"], case["T"], case["D"]
    if op == "dropout":
        return {"bytes": T * D * _BYTES[case["dtype"]] * (3 if case["residual"] else 2), "flops": 2 * T * D}
    if op.startswith("layer"):
        r, p, b = _BYTES[case["residual"]], _BYTES[case["params"]], 2 if case["branch"] else 0
        if op == "layer_norm_forward":      # x, branch -> y, h
            return {"bytes": T * D * (2 * r + b + 2) + 2 * D * p + 8 * T, "flops": 10 * T * D}
        # y, dy, dh -> dx, dbranch and the parameters' gradients
        return {"bytes": T * D * (3 * r + 2 + b) + D * p + 8 * D + 8 * T, "flops": 20 * T * D}
    V, n = case["V"], T - case["ignored"]
    if op == "cross_entropy_forward":
        return {"bytes": 2 * V * D + 2 * n * D + 16 * T, "flops": 2 * n * V * D}
    # the logits again, the gradients of h and of the weights
    return {"bytes": 4 * V * D + 2 * n * D + 2 * T * D + 16 * T, "flops": 6 * n * V * D}


# ---------------------------------------------------------- in 64 bits

def _exact_keep(s):
    """The dropout's factors, from the generator's definition on 64-bit words."""
    c = s["case"]
    n = c["T"] * c["D"]
    seed, step = (int(v) for v in s["rng"].cpu())
    m32 = np.uint64(0xFFFFFFFF)
    ctr = [np.arange((n + 7) // 8, dtype=np.uint64) & m32, np.arange((n + 7) // 8, dtype=np.uint64) >> np.uint64(32),
           np.uint64(SITE), np.uint64(step & 0xFFFFFFFF)]
    key = [seed & 0xFFFFFFFF, (seed >> 32) & 0xFFFFFFFF]
    for _ in range(10):
        a, b = ctr[0] * np.uint64(0xD2511F53), ctr[2] * np.uint64(0xCD9E8D57)
        ctr = [(b >> np.uint64(32)) ^ ctr[1] ^ np.uint64(key[0]), b & m32,
               (a >> np.uint64(32)) ^ ctr[3] ^ np.uint64(key[1]), a & m32]
        key = [(key[0] + 0x9E3779B9) & 0xFFFFFFFF, (key[1] + 0xBB67AE85) & 0xFFFFFFFF]
    words = np.stack(ctr, 1).astype("<u4").view("<u2").reshape(-1)[:n]
    t = _threshold(c["p"])
    keep = torch.from_numpy(words >= t).to(s["rng"].device).view(c["T"], c["D"])
    return keep, 65536.0 / (65536 - t)


def _exact_dropped(s, x):
    if s["case"]["p"] == 0.0:
        return x
    keep, scale = _exact_keep(s)
    return (x * scale).masked_fill(~keep, 0.0)


def _exact_norm(case, s):
    if case["op"] == "layer_norm_forward":
        y = ALPHA * s["x"].double()
        if case["branch"]:
            y = y + BETA * _exact_dropped(s, s["branch"].double())
        var, mean = torch.var_mean(y, 1, correction=0)
        h = torch.addcmul(s["bias"].double(), (y - mean[:, None]) * (var[:, None] + EPS) ** -0.5, s["weight"].double())
        return {"y": y, "h": h, "stats": torch.stack((mean, (var + EPS) ** -0.5))}
    y = s["y"].double().requires_grad_(True)
    w = s["weight"].double().requires_grad_(True)
    b = s["bias"].double().requires_grad_(True)
    var, mean = torch.var_mean(y, 1, correction=0, keepdim=True)
    h = (y - mean) * (var + EPS) ** -0.5 * w + b
    dy, dw, db = torch.autograd.grad((h, y), (y, w, b), (s["dh"].double(), s["dy"].double()))
    out = {"dx": ALPHA * dy, "dweight": dw, "dbias": db}
    if case["branch"]:
        out["dbranch"] = BETA * _exact_dropped(s, dy)
    return out


def _exact_ce(case, s):
    T, D, V = case["T"], case["D"], case["V"]
    forward = case["op"] == "cross_entropy_forward"
    if (2 if forward else 6) * T * D * V > 8e12:
        return None
    rows = torch.nonzero(s["targets"] != IGNORE)[:, 0]
    h, t = s["h"][rows].double(), s["targets"][rows]
    hit = (h * s["weight"][t].double()).sum(1)
    step = max(256, (1 << 28) // max(1, len(rows)))
    if forward:
        parts = [torch.logsumexp(h @ s["weight"][v:v + step].double().t(), 1) for v in range(0, V, step)]
        lse = torch.logsumexp(torch.stack(parts), 0)
        out = torch.zeros((2, T), dtype=torch.float64, device=h.device)
        out[0, rows] = lse - hit + case["z"] * lse ** 2
        out[1, rows] = lse
        return {"loss": out[0], "lse": out[1]}
    lse, d = s["lse"][rows].double(), s["d_loss"][rows].double()
    dh = torch.zeros((T, D), dtype=torch.float64, device=h.device)
    dweight = torch.empty((V, D), dtype=torch.float64, device=h.device)
    share = d * (1.0 + 2.0 * case["z"] * lse)
    grad = torch.zeros((len(rows), D), dtype=torch.float64, device=h.device)
    for v in range(0, V, step):
        w = s["weight"][v:v + step].double()
        p = torch.exp(h @ w.t() - lse[:, None]) * share[:, None]
        grad += p @ w
        dweight[v:v + step] = p.t() @ h
    dh[rows] = grad - d[:, None] * s["weight"][t].double()
    dweight.index_add_(0, t, -d[:, None] * h)
    return {"dh": dh, "dweight": dweight}


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "dropout":
        x = _exact_dropped(s, s["x"].double())
        return x if s["residual"] is None else x + s["residual"].double()
    if case["op"].startswith("layer"):
        return _exact_norm(case, s)
    return _exact_ce(case, s)
