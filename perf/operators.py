"""Timed cases of the operators around the routed experts, and their plain forms.

Three operators of a training or serving step, next to the routed layer:

* ``norm``: the norm after a block, its gate, the scaled residual and the norm
  before the next block in one pass,
      p = branch * rsqrt(mean(branch^2) + eps) * (post_weight + offset)
      y = residual_scale * x + branch_scale * gate * p
      h = y * rsqrt(mean(y^2) + eps) * (pre_weight + offset)
  and its backward pass (gradients of x, branch, the gate and both weights);
* ``gate``: the router's choice of top_k experts a token from its logits, with
  the scores of the chosen ones, and the gradient of the logits;
* ``muon``: updates of stacked expert weights [E, N, K] made orthogonal by
  Newton-Schulz products, X <- a X + (b A + c A A) X with A = X X^T, from
  X = U / (|U| + eps), alone or as the whole optimiser step (momentum,
  Nesterov mix, weight decay, update).

``run`` computes a case in its plain form (elementary torch operations in 32
bits, rounded once at the end) or, with ``own``, through the framework.
Sizes are those of the framework's workloads (D = 256, 2048, 7168; F = 512,
1408, 2048; E = 8, 64, 384; top_k = 2, 6, 8) and odd ones.
"""

import math

import numpy as np
import torch

own = False

COEFFICIENTS = (3.4445, -4.7750, 2.0315)
STEPS = 5
NORM_EPS = 1e-6
MUON_EPS = 1e-7
MU = 0.95
SIGMOID_EPS = 1e-20

_TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
_BYTES = {"bf16": 2, "fp32": 4}


# -------------------------------------------------------------------- cases

def _norm(name, op, T, D, residual, gate, groups=1, params="bf16"):
    c = {"op": op, "T": T, "D": D, "residual": residual, "gate": gate, "groups": groups, "params": params}
    return dict(c, name=name) if name else c


def _gate(name, op, T, E, K, dtype, score, renormalize, bias, masked):
    c = {"op": op, "T": T, "E": E, "K": K, "dtype": dtype, "score": score, "renormalize": renormalize, "bias": bias,
         "masked": masked}
    return dict(c, name=name) if name else c


def _orth(name, E, N, K, dtype):
    c = {"op": "orthogonalize", "E": E, "N": N, "K": K, "dtype": dtype}
    return dict(c, name=name) if name else c


def _muon(name, E, N, K, weight, lr):
    c = {"op": "muon_update", "E": E, "N": N, "K": K, "weight": weight, "lr": lr}
    return dict(c, name=name) if name else c


def listed():
    return [
        # one decode token between two blocks of the E=384 model: latency
        _norm("norm decode 1x7168", "norm_forward", 1, 7168, "bf16", "channel"),
        # the E=384 training step's tokens, statistics kept for the backward
        _norm("norm forward 2048x7168", "norm_forward", 2048, 7168, "bf16", "channel"),
        # a long packed batch of the D=2048 model with an FP32 residual stream and one gate row a sequence
        _norm("norm forward 16384x2048", "norm_forward", 16384, 2048, "fp32", "group", 8),
        # the E=384 training step's backward
        _norm("norm backward 2048x7168", "norm_backward", 2048, 7168, "bf16", "channel"),
        # a ragged batch and a width that no vector divides, one gate value a token
        _norm("norm backward 1531x1411", "norm_backward", 1531, 1411, "fp32", "token", 1, "fp32"),
        # one decode token's choice among 384 experts
        _gate("gate forward 1x384", "gate_forward", 1, 384, 6, "fp32", "softmax", True, False, False),
        # a training step's tokens, sigmoid scores with a selection bias, masked experts and tokens
        _gate("gate forward 16384x384", "gate_forward", 16384, 384, 8, "fp32", "sigmoid", True, True, True),
        # its backward where the scores are shares of all experts: every logit has a gradient
        _gate("gate backward 4096x384", "gate_backward", 4096, 384, 6, "fp32", "softmax", False, False, True),
        # the smallest workload's expert weights: launches count
        _orth("orthogonalize 8x512x256", 8, 512, 256, "bf16"),
        # FP32 gradients whose sizes no tile divides
        _orth("orthogonalize 3x1000x1531", 3, 1000, 1531, "fp32"),
        # eight experts' W2 gradients (taller than wide) of the E=384 layer
        _orth("orthogonalize 8x7168x2048", 8, 7168, 2048, "bf16"),
        # the whole step on the gate projections of the E=64 layer, FP32 master weights
        _muon("muon update 64x1408x2048", 64, 1408, 2048, "fp32", 1e-4),
    ]


def _log(rng, lo, hi):
    n = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    return n + 1 if n == 3072 else n


def _products(N, K):
    """Multiply-adds x 2 of one Newton-Schulz step's three products: A and the
    polynomial are symmetric, so half of each is enough."""
    m, k = min(N, K), max(N, K)
    return m * (m + 1) * k + m * (m + 1) * m + 2 * m * m * k


def draw(rng):
    op = rng.choice(["norm_forward", "norm_backward", "gate_forward", "gate_backward", "orthogonalize", "muon_update"])
    if op.startswith("norm"):
        D = rng.choice([256, 2048, 7168, _log(rng, 64, 8192), 16 * (_log(rng, 8, 512) | 1)])
        T = _log(rng, 1, max(1, min(16384, 2048 * 7168 // D)))
        gate = rng.choice(["none", "channel", "group", "token", "full"])
        groups = 1
        if gate == "group":
            groups = rng.choice([2, 3, 8])
            T = groups * max(1, T // groups)
        return _norm(None, op, T, D, rng.choice(["bf16", "fp32"]), gate, groups, rng.choice(["bf16", "fp32"]))
    if op.startswith("gate"):
        E = rng.choice([8, 64, 384, _log(rng, 8, 1024)])
        K = rng.randint(1, min(E, rng.choice([2, 8, 32])))
        return _gate(None, op, _log(rng, 1, min(32768, 16384 * 384 // E)), E, K, rng.choice(["fp32", "bf16"]),
                     rng.choice(["softmax", "sigmoid"]), K > 1 and rng.random() < 0.5, rng.random() < 0.5,
                     rng.random() < 0.5)
    N, K = _log(rng, 48, 2048), rng.choice([_log(rng, 48, 2816), 2048, 7168])
    if rng.random() < 0.5:
        N = max(1, N // 64) * 64
    if rng.random() < 0.5:
        N, K = K, N
    most = 64 * _products(1408, 2048)
    E = _log(rng, 1, max(1, min(64, most // (2 * _products(N, K)))))
    if op == "orthogonalize":
        return _orth(None, E, N, K, rng.choice(["bf16", "fp32"]))
    return _muon(None, E, N, K, rng.choice(["fp32", "bf16"]), round(10 ** rng.uniform(-5, -4), 7))


# ------------------------------------------------------------------- inputs

def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    rnd = lambda *shape: torch.randn(shape, generator=g, device=dev)  # noqa: E731
    s = {"case": case}
    op = case["op"]
    if op.startswith("norm"):
        T, D = case["T"], case["D"]
        res, par = _TYPES[case["residual"]], _TYPES[case["params"]]
        # a residual stream grows over the layers and has a few large channels
        channels = torch.where(torch.rand(D, generator=g, device=dev) < 0.01, 20.0, 1.0)
        s["x"] = (2.0 * channels * rnd(T, D)).to(res)
        s["branch"] = (0.3 * rnd(T, D)).to(torch.bfloat16)
        s["post_weight"] = (1.0 + 0.1 * rnd(D)).to(par)
        s["pre_weight"] = (1.0 + 0.1 * rnd(D)).to(par)
        shape = {"none": None, "channel": (D,), "group": (case["groups"], D), "token": (T, 1), "full": (T, D)}[case["gate"]]
        s["gate"] = None if shape is None else (0.5 + 0.2 * rnd(*shape)).to(par)
        s["scales"] = {"residual_scale": 0.95, "branch_scale": 0.7}
        if op == "norm_backward":
            s["dy"] = rnd(T, D).to(res)
            s["dh"] = rnd(T, D).to(torch.bfloat16)
            x, b = s["x"].float(), s["branch"].float()
            rp = torch.rsqrt((b * b).mean(1) + NORM_EPS)
            p = b * rp[:, None] * s["post_weight"].float()
            if s["gate"] is not None:
                p = p * _gate_rows(s["gate"].float(), T)
            y = 0.95 * x + 0.7 * p
            # what the forward pass saved
            s["stats"] = torch.stack((rp, torch.rsqrt((y * y).mean(1) + NORM_EPS)))
    elif op.startswith("gate"):
        T, E, K = case["T"], case["E"], case["K"]
        # a router's logits: some experts are popular, and BF16 logits have ties
        logits = rnd(T, E) * 1.5 + rnd(E)
        if case["masked"]:
            logits = logits.masked_fill(torch.rand((T, E), generator=g, device=dev) < 0.1, -math.inf)
            empty = torch.rand(T, generator=g, device=dev) < 0.03     # padding tokens: every expert masked
            logits = logits.masked_fill(empty[:, None], -math.inf)
        s["logits"] = logits.to(_TYPES[case["dtype"]])
        s["bias"] = 0.3 * rnd(E) if case["bias"] else None
        s["scale"] = 2.5
        if op == "gate_backward":
            s["ids"] = _choose(s["logits"], s["bias"], K)[0]
            s["d_scores"] = rnd(T, K)
    else:
        E, N, K = case["E"], case["N"], case["K"]
        # an expert's gradient: a few strong directions from its tokens over a
        # weak full-rank part; experts that no token reached have none
        r = min(32, N, K)
        decay = torch.logspace(0, -2, r, device=dev)
        grad = torch.empty((E, N, K), device=dev, dtype=torch.float32)
        for e in range(E):
            grad[e] = 1e-3 * ((rnd(N, r) * decay) @ rnd(r, K) + 0.02 * rnd(N, K))
        if E > 4:
            grad[E // 2] = 0.0
        if op == "orthogonalize":
            s["x"] = grad.to(_TYPES[case["dtype"]])
        else:
            s["grad"] = grad.to(torch.bfloat16)
            s["momentum"] = grad
            for e in range(E):
                s["momentum"][e] += 1e-3 * (rnd(N, r) @ rnd(r, K)) * 0.3
            s["weight"] = torch.empty((E, N, K), device=dev, dtype=_TYPES[case["weight"]])
            for e in range(E):
                s["weight"][e] = (rnd(N, K) * K ** -0.5).to(s["weight"].dtype)
            s["copy"] = torch.empty((E, N, K), device=dev, dtype=torch.bfloat16) if case["weight"] == "fp32" else None
            s["scale"] = 0.2 * math.sqrt(max(N, K))
    return s


# -------------------------------------------------------------- plain forms

def _gate_rows(gate, T):
    """A gate [D], [G, D], [T, 1] or [T, D] as rows [T, D] (or broadcast)."""
    if gate.dim() == 1:
        return gate[None]
    return gate if gate.shape[0] == T else gate.repeat_interleave(T // gate.shape[0], 0)


def _norm_forward(s):
    c = s["case"]
    T = c["T"]
    x, b = s["x"].float(), s["branch"].float()
    rp = torch.rsqrt((b * b).mean(1, keepdim=True) + NORM_EPS)
    p = b * rp * s["post_weight"].float()
    if s["gate"] is not None:
        p = p * _gate_rows(s["gate"].float(), T)
    y = s["scales"]["residual_scale"] * x + s["scales"]["branch_scale"] * p
    ry = torch.rsqrt((y * y).mean(1, keepdim=True) + NORM_EPS)
    h = y * ry * s["pre_weight"].float()
    return {"y": y.to(s["x"].dtype), "h": h.to(torch.bfloat16), "stats": torch.cat((rp, ry), 1).t()}


def _norm_backward(s):
    c = s["case"]
    T = c["T"]
    alpha, beta = s["scales"]["residual_scale"], s["scales"]["branch_scale"]
    x, b = s["x"].float(), s["branch"].float()
    dy, dh = s["dy"].float(), s["dh"].float()
    wp, wh = s["post_weight"].float(), s["pre_weight"].float()
    rp, ry = s["stats"][0][:, None], s["stats"][1][:, None]
    n = b * rp
    p = n * wp
    gate = None if s["gate"] is None else _gate_rows(s["gate"].float(), T)
    gp = p if gate is None else p * gate
    yn = (alpha * x + beta * gp) * ry
    out = {"dpre_weight": (dh * yn).sum(0)}
    dn = dh * wh
    ds = dy + ry * (dn - yn * (dn * yn).mean(1, keepdim=True))
    out["dx"] = (alpha * ds).to(s["x"].dtype)
    if gate is not None:
        dg = beta * ds * p
        if c["gate"] == "channel":
            dg = dg.sum(0)
        elif c["gate"] == "group":
            dg = dg.view(c["groups"], -1, dg.shape[1]).sum(1)
        elif c["gate"] == "token":
            dg = dg.sum(1, keepdim=True)
        out["dgate"] = dg.to(s["gate"].dtype)
    dp = beta * ds if gate is None else beta * ds * gate
    out["dpost_weight"] = (dp * n).sum(0)
    dn = dp * wp
    out["dbranch"] = (rp * (dn - n * (dn * n).mean(1, keepdim=True))).to(torch.bfloat16)
    return out


def _choose(logits, bias, K):
    """(ids, chosen): the top_k keys of each row, equal keys by index; -1 where none is left."""
    key = logits.float() if bias is None else logits.float() + bias
    top, ids = torch.sort(key, dim=1, descending=True, stable=True)
    chosen = top[:, :K] > -math.inf
    return torch.where(chosen, ids[:, :K], -1).to(torch.int32), chosen


def _scores(s, logits, ids, chosen):
    """The chosen scores before the scale, the sigmoids' slopes, and what the scores were divided by."""
    c = s["case"]
    l = torch.gather(logits, 1, ids.clamp(min=0).long())
    if c["score"] == "sigmoid":
        v = torch.where(chosen, 1.0 / (1.0 + torch.exp(-l)), 0.0)
        total = v.sum(1, keepdim=True) + SIGMOID_EPS
        return (v / total if c["renormalize"] else v), v / (1.0 + torch.exp(l)), total
    if c["renormalize"]:
        l = torch.where(chosen, l, -math.inf)
        top = l.max(1, keepdim=True).values
        v = torch.where(chosen, torch.exp(l - top), 0.0)
        total = v.sum(1, keepdim=True)
    else:
        top = logits.max(1, keepdim=True).values
        total = torch.exp(logits - top).sum(1, keepdim=True)
        v = torch.where(chosen, torch.exp(l - top), 0.0)
    total = torch.where(total > 0, total, 1.0)      # rows without experts
    return v / total, None, total


def _gate_forward(s):
    ids, chosen = _choose(s["logits"], s["bias"], s["case"]["K"])
    return {"ids": ids, "scores": s["scale"] * _scores(s, s["logits"].float(), ids, chosen)[0]}


def _gate_backward(s):
    c = s["case"]
    ids = s["ids"]
    chosen = ids >= 0
    logits = s["logits"].float()
    d = s["scale"] * torch.where(chosen, s["d_scores"], 0.0)
    sc, slope, total = _scores(s, logits, ids, chosen)
    if c["score"] == "sigmoid":
        if c["renormalize"]:
            d = (d - (d * sc).sum(1, keepdim=True)) / total
        dl = d * slope
    else:
        dl = sc * d
        if c["renormalize"]:
            dl = dl - sc * dl.sum(1, keepdim=True)
    out = torch.zeros_like(logits)
    out.scatter_add_(1, ids.clamp(min=0).long(), torch.where(chosen, dl, 0.0))
    if c["score"] == "softmax" and not c["renormalize"]:
        top = logits.max(1, keepdim=True).values
        share = torch.where(top > -math.inf, torch.exp(logits - top) / total, 0.0)
        out = out - share * dl.sum(1, keepdim=True)
    return out.to(s["logits"].dtype)


def _newton_schulz(u):
    x = u / (torch.sqrt((u * u).sum((1, 2), keepdim=True)) + MUON_EPS)
    tall = x.shape[1] > x.shape[2]
    if tall:
        x = x.transpose(1, 2)
    a, b, c = COEFFICIENTS
    for _ in range(STEPS):
        xx = torch.matmul(x, x.transpose(1, 2))
        x = a * x + torch.matmul(b * xx + c * torch.matmul(xx, xx), x)
    return x.transpose(1, 2) if tall else x


def _muon_update(s):
    grad = s["grad"].float()
    s["momentum"].mul_(MU).add_(grad)
    o = _newton_schulz(grad + MU * s["momentum"])
    lr = s["case"]["lr"]
    w = s["weight"].float() * (1.0 - lr * 0.1) - (lr * s["scale"]) * o
    s["weight"].copy_(w)
    if s["copy"] is not None:
        s["copy"].copy_(w)
    return {"weight": s["weight"], "momentum": s["momentum"], "copy": s["copy"]}


def _plain(s):
    op = s["case"]["op"]
    if op == "norm_forward":
        return _norm_forward(s)
    if op == "norm_backward":
        return _norm_backward(s)
    if op == "gate_forward":
        return _gate_forward(s)
    if op == "gate_backward":
        return _gate_backward(s)
    if op == "orthogonalize":
        return _newton_schulz(s["x"].float()).to(torch.bfloat16)
    return _muon_update(s)


# ------------------------------------------------------------ the framework

def _framework(s):
    from mixture_experts_routed_route_gb300 import block, optim
    c = s["case"]
    op = c["op"]
    if op == "norm_forward":
        stats = torch.empty((2, c["T"]), dtype=torch.float32, device=s["x"].device)
        y, h = block.block_norm(s["x"], s["branch"], gate=s["gate"], post_weight=s["post_weight"],
                                pre_weight=s["pre_weight"], eps=NORM_EPS, stats=stats, **s["scales"])
        return {"y": y, "h": h, "stats": stats}
    if op == "norm_backward":
        r = block.block_norm_backward(s["x"], s["branch"], s["stats"], s["dy"], s["dh"], gate=s["gate"],
                                      post_weight=s["post_weight"], pre_weight=s["pre_weight"], **s["scales"])
        out = {"dx": r.dx, "dbranch": r.dbranch, "dpost_weight": r.dpost_weight, "dpre_weight": r.dpre_weight}
        if s["gate"] is not None:
            out["dgate"] = r.dgate
        return out
    if op == "gate_forward":
        ids, scores = block.topk_gate(s["logits"], c["K"], score=c["score"], renormalize=c["renormalize"],
                                      scale=s["scale"], select_bias=s["bias"])
        return {"ids": ids, "scores": scores}
    if op == "gate_backward":
        return block.topk_gate_backward(s["logits"], s["ids"], s["d_scores"], score=c["score"],
                                        renormalize=c["renormalize"], scale=s["scale"])
    if op == "orthogonalize":
        return optim.orthogonalize(s["x"], steps=STEPS, coefficients=COEFFICIENTS, eps=MUON_EPS)
    optim.muon_update(s["weight"], s["grad"], s["momentum"], lr=c["lr"], mu=MU, nesterov=True, weight_decay=0.1,
                      scale=s["scale"], steps=STEPS, coefficients=COEFFICIENTS, eps=MUON_EPS, weight_bf16=s["copy"])
    return {"weight": s["weight"], "momentum": s["momentum"], "copy": s["copy"]}


def run(state):
    return _framework(state) if own else _plain(state)


# --------------------------------------------------------------------- work

def work(case):
    op = case["op"]
    if op.startswith("norm"):
        T, D, r, p = case["T"], case["D"], _BYTES[case["residual"]], _BYTES[case["params"]]
        gate = {"none": 0, "channel": D, "group": case["groups"] * D, "token": T, "full": T * D}[case["gate"]] * p
        if op == "norm_forward":      # x, branch -> y, h
            return {"bytes": T * D * (2 * r + 4) + gate + 2 * D * p + 8 * T, "flops": 10 * T * D}
        # x, branch, dy, dh -> dx, dbranch and the parameters' gradients
        return {"bytes": T * D * (3 * r + 6) + 2 * gate + 2 * D * p + 8 * D + 8 * T, "flops": 30 * T * D}
    if op.startswith("gate"):
        T, E, K, b = case["T"], case["E"], case["K"], _BYTES[case["dtype"]]
        if op == "gate_forward":
            return {"bytes": T * E * b + T * K * 8 + (4 * E if case["bias"] else 0), "flops": T * E * 4}
        read = T * E * b if case["score"] == "softmax" and not case["renormalize"] else T * K * b
        return {"bytes": read + T * E * b + T * K * 8, "flops": T * E * 4}
    E, N, K = case["E"], case["N"], case["K"]
    flops = E * STEPS * _products(N, K)
    if op == "orthogonalize":
        return {"bytes": E * N * K * (_BYTES[case["dtype"]] + 2), "flops": flops}
    w = _BYTES[case["weight"]]
    return {"bytes": E * N * K * (2 + 8 + 2 * w + (2 if w == 4 else 0)), "flops": flops}


# ---------------------------------------------------------- in 64 bits

def _exact_norm(case, s):
    T = case["T"]
    names = ["x", "branch", "post_weight", "pre_weight"] + (["gate"] if s["gate"] is not None else [])
    v = {n: s[n].double().requires_grad_(True) for n in names}

    def rms(t):
        return ((t ** 2).sum(-1) / t.shape[-1] + NORM_EPS) ** -0.5

    after = rms(v["branch"])
    block = torch.einsum("td,t,d->td", v["branch"], after, v["post_weight"])
    if s["gate"] is not None:
        if case["gate"] == "group":
            block = (block.reshape(case["groups"], -1, case["D"]) * v["gate"][:, None]).reshape(T, -1)
        else:
            block = block * v["gate"]
    y = s["scales"]["residual_scale"] * v["x"] + s["scales"]["branch_scale"] * block
    before = rms(y)
    h = torch.einsum("td,t,d->td", y, before, v["pre_weight"])
    if case["op"] == "norm_forward":
        return {"y": y.detach(), "h": h.detach(), "stats": torch.stack((after, before)).detach()}
    grads = torch.autograd.grad((y, h), list(v.values()), (s["dy"].double(), s["dh"].double()))
    return {"d" + n: g for n, g in zip(v, grads)}


def _exact_gate(case, s):
    logits = s["logits"].double()
    leaf = logits.clone().requires_grad_(True)
    K = case["K"]
    if case["op"] == "gate_backward":
        ids = s["ids"].long()
    else:
        key = s["logits"].float().cpu().numpy()
        if s["bias"] is not None:
            key = key + s["bias"].cpu().numpy()      # the choice is made on FP32 sums
        order = np.argsort(-key, axis=1, kind="stable")[:, :K]
        left = np.take_along_axis(key, order, 1) > -np.inf
        ids = torch.from_numpy(np.where(left, order, -1)).to(logits.device)
    on = torch.zeros_like(logits, dtype=torch.bool)
    on.scatter_(1, ids.clamp(min=0), True)
    none = (ids < 0).all(1)
    on = on & ~none[:, None]
    # index 0 was marked by the -1 of a row that has fewer than K experts
    first = (ids == 0).any(1)
    on[:, 0] = on[:, 0] & first
    if case["score"] == "sigmoid":
        all_scores = torch.sigmoid(leaf)
        if case["renormalize"]:
            all_scores = all_scores / (torch.where(on, all_scores, 0.0).sum(1, keepdim=True) + SIGMOID_EPS)
    else:
        kept = on if case["renormalize"] else logits > -math.inf
        safe = torch.where(kept, leaf, -1e300)
        shifted = torch.where(kept, torch.exp(safe - safe.max(1, keepdim=True).values.detach()), 0.0)
        all_scores = shifted / shifted.sum(1, keepdim=True).clamp(min=1e-300)
    all_scores = s["scale"] * torch.where(on, all_scores, 0.0)
    scores = torch.where(ids >= 0, torch.gather(all_scores, 1, ids.clamp(min=0)), 0.0)
    if case["op"] == "gate_forward":
        return {"ids": None, "scores": scores.detach()}
    return torch.autograd.grad(scores, leaf, s["d_scores"].double())[0]


def _exact_muon(case, s):
    if case["E"] * STEPS * 2 * _products(case["N"], case["K"]) > 1.6e13:
        return None
    if case["op"] == "orthogonalize":
        u = s["x"]
    else:
        momentum = MU * s["momentum"].double() + s["grad"].double()
        u = momentum
    a, b, c = COEFFICIENTS
    o = torch.empty(u.shape, dtype=torch.float64, device=u.device)
    for e in range(case["E"]):
        x = u[e].double()
        if case["op"] == "muon_update":
            x = s["grad"][e].double() + MU * x
        x = x / (torch.linalg.vector_norm(x) + MUON_EPS)
        for _ in range(STEPS):
            # the polynomial on whichever side is the smaller one
            if x.shape[0] <= x.shape[1]:
                q = x @ x.T
                x = a * x + b * (q @ x) + c * (q @ (q @ x))
            else:
                q = x.T @ x
                x = a * x + b * (x @ q) + c * ((x @ q) @ q)
        o[e] = x
    if case["op"] == "orthogonalize":
        return o
    w = s["weight"].double() * (1.0 - case["lr"] * 0.1) - case["lr"] * s["scale"] * o
    return {"weight": w, "momentum": momentum, "copy": w if s["copy"] is not None else None}


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"].startswith("norm"):
        return _exact_norm(case, s)
    if case["op"].startswith("gate"):
        return _exact_gate(case, s)
    return _exact_muon(case, s)
