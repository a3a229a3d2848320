"""Workloads of the router and of the dense products around the experts.

What is timed here, with the plain form of each operator beside the call a
user makes of it:

* ``route``       -- a token's experts and their weights from its logits:
  softmax or sigmoid scores, a bias for balance, groups, top-k, renormalised
  weights;
* ``route_grad``  -- the gradient of those weights, for the logits;
* ``linear``      -- a product with bias, activation and residual: the router's
  logits, a shared expert's gate-up and down products;
* ``linear_grad`` -- its gradients: of the input, the weight and the bias.

``T`` tokens, ``E`` experts, ``K`` experts per token; a product takes rows of
``H`` values to ``N`` (swiglu: to 2N, a gate half and an up half, joined to N).
"""
import math

import torch

own = False

BF16, F32, F64 = torch.bfloat16, torch.float32, torch.float64
INF = float("inf")

# The largest draws stay within these: bytes moved and operations of one pass.
MOST_BYTES = 1.5e9
MOST_FLOPS = 4.8e11


def listed():
    return [
        # One new token of the DeepSeek-V3-shaped router: sigmoid scores, a bias
        # that keeps the experts' load even, four of eight groups.
        {"name": "route one token", "op": "route", "T": 1, "E": 256, "K": 8, "score": "sigmoid",
         "bias": True, "groups": 8, "topk_groups": 4, "group_score": "top2", "renorm": True,
         "scale": 2.5, "type": "f32", "masked": 0.0},
        # A long prefill through the same router.
        {"name": "route long prefill", "op": "route", "T": 16384, "E": 256, "K": 8,
         "score": "sigmoid", "bias": True, "groups": 8, "topk_groups": 4, "group_score": "top2",
         "renorm": True, "scale": 2.5, "type": "f32", "masked": 0.0},
        # Softmax scores over a number of experts that fills no warp, bf16
        # logits (equal ones are common), experts taken out for some tokens and
        # padding tokens without any.
        {"name": "route softmax odd", "op": "route", "T": 4999, "E": 60, "K": 4, "score": "softmax",
         "bias": False, "groups": 1, "topk_groups": 1, "group_score": "max", "renorm": False,
         "scale": 1.0, "type": "bf16", "masked": 0.2},
        # The prefill router's training step.
        {"name": "route_grad prefill", "op": "route_grad", "T": 4096, "E": 256, "K": 8,
         "score": "sigmoid", "renorm": True, "scale": 2.5, "type": "f32", "masked": 0.0},
        # A dense gradient: softmax weights that are not renormalised reach
        # every logit.
        {"name": "route_grad dense", "op": "route_grad", "T": 16383, "E": 128, "K": 8,
         "score": "softmax", "renorm": False, "scale": 1.0, "type": "f32", "masked": 0.1},
        # The router's logits of a decode batch: one tile of output, a long sum.
        {"name": "linear logits decode", "op": "linear", "T": 128, "H": 7168, "N": 256,
         "bias": False, "act": "none", "residual": False, "out": "f32", "keep_z": False},
        # The same of a long prefill: bound by reading the rows.
        {"name": "linear logits prefill", "op": "linear", "T": 16384, "H": 7168, "N": 256,
         "bias": False, "act": "none", "residual": False, "out": "f32", "keep_z": False},
        # A shared expert's gate-up product for one new token: the time is that
        # of reading the weights.
        {"name": "linear gate-up one token", "op": "linear", "T": 1, "H": 7168, "N": 2048,
         "bias": False, "act": "swiglu", "residual": False, "out": "bf16", "keep_z": False},
        # Its down product over a long prefill, added to the routed experts'
        # result: bound by the tensor cores.
        {"name": "linear down prefill", "op": "linear", "T": 16384, "H": 2048, "N": 7168,
         "bias": False, "act": "none", "residual": True, "out": "bf16", "keep_z": False},
        # Odd everything, with all of the epilogue, as a training step calls it.
        {"name": "linear odd", "op": "linear", "T": 333, "H": 1000, "N": 1075, "bias": True,
         "act": "gelu", "residual": True, "out": "bf16", "keep_z": True},
        # The shared expert's gate-up product in a training step.
        {"name": "linear_grad gate-up", "op": "linear_grad", "T": 4096, "H": 7168, "N": 2048,
         "bias": False, "act": "swiglu", "dy": "bf16"},
        # The router's product in a training step, from the logits' gradient.
        {"name": "linear_grad logits", "op": "linear_grad", "T": 4095, "H": 2048, "N": 60,
         "bias": True, "act": "none", "dy": "f32"},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    while True:
        op = rng.choice(["route", "route_grad", "linear", "linear_grad"])
        if op in ("route", "route_grad"):
            groups = rng.choice([1, 1, 4, 8]) if op == "route" else 1
            E = groups * _log_int(rng, 8 if groups == 1 else 2, 512 // groups)
            most = max(1, groups // 2)
            c = {"op": op, "T": _log_int(rng, 1, 16384), "E": E,
                 "K": rng.randint(1, min(8, E // groups * most)),
                 "score": rng.choice(["softmax", "sigmoid"]), "renorm": rng.choice([False, True]),
                 "scale": rng.choice([1.0, 2.5]), "type": rng.choice(["f32", "bf16"]),
                 "masked": rng.choice([0.0, 0.0, 0.1, 0.5])}
            if op == "route":
                c.update(bias=rng.choice([False, True]), groups=groups, topk_groups=most,
                         group_score=rng.choice(["max", "top2"]))
        else:
            c = {"op": op, "T": _log_int(rng, 1, 16384), "H": 8 * _log_int(rng, 8, 1024),
                 "N": _log_int(rng, 8, 8192), "bias": rng.choice([False, True]),
                 "act": rng.choice(["none", "none", "relu", "gelu", "silu", "swiglu"])}
            if op == "linear":
                c.update(residual=rng.choice([False, True]), out=rng.choice(["bf16", "f32"]),
                         keep_z=rng.choice([False, True]))
            else:
                c.update(dy=rng.choice(["bf16", "f32"]))
        w = work(c)
        if w["bytes"] <= MOST_BYTES and w["flops"] <= MOST_FLOPS:
            return c


# -- inputs -------------------------------------------------------------------

_TYPES = {"bf16": BF16, "f32": F32}


def _logits(c, g):
    """[T, E] as a router's product leaves them: some experts more popular than
    others, some entries taken out, and padding tokens without any."""
    l = torch.randn((c["T"], c["E"]), generator=g, device="cuda")
    l += 0.7 * torch.randn(c["E"], generator=g, device="cuda")
    if c["masked"]:
        l[torch.rand(l.shape, generator=g, device="cuda") < c["masked"]] = -INF
        l[torch.rand(c["T"], generator=g, device="cuda") < c["masked"] / 4] = -INF
    return l.to(_TYPES[c["type"]])


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed) * 7919 + 31)
    s = {"case": c}

    def randn(*shape, dtype=BF16):
        return torch.randn(shape, generator=g, device="cuda", dtype=dtype)

    def empty(*shape, dtype=BF16):
        return torch.empty(shape, dtype=dtype, device="cuda")

    T = c["T"]
    if c["op"] in ("route", "route_grad"):
        E, K = c["E"], c["K"]
        s["logits"] = _logits(c, g)
        if c["op"] == "route":
            # as large as the scores' differences that it is there to outweigh
            size = 0.1 if c["score"] == "sigmoid" else 0.5 / E
            s["bias"] = size * randn(E, dtype=F32) if c["bias"] else None
            s["topk_idx"] = empty(T, K, dtype=torch.int64)
            s["topk_w"] = empty(T, K, dtype=F32)
        else:
            top, idx = s["logits"].float().sort(dim=1, descending=True, stable=True)
            s["topk_idx"] = torch.where(top > -INF, idx, -1)[:, :K].contiguous()
            s["d_topk_w"] = randn(T, K, dtype=F32)
            s["d_logits"] = torch.empty_like(s["logits"])
        return s
    H, N = c["H"], c["N"]
    wide = 2 * N if c["act"] == "swiglu" else N
    s["x"] = randn(T, H)
    s["w"] = randn(wide, H) * H ** -0.5
    if c["op"] == "linear":
        out = _TYPES[c["out"]]
        s["bias"] = 0.1 * randn(wide, dtype=F32) if c["bias"] else None
        s["residual"] = randn(T, N, dtype=out) if c["residual"] else None
        s["z"] = empty(T, wide) if c["keep_z"] else None
        s["y"] = empty(T, N, dtype=out)
        return s
    s["dy"] = randn(T, N, dtype=_TYPES[c["dy"]])
    s["z"] = randn(T, wide) if c["act"] != "none" else None
    # rows of dz start on 16 bytes
    s["dz"] = empty(T, -(-wide // 8) * 8)
    s["dx"], s["d_w"] = empty(T, H), empty(wide, H)
    s["d_bias"] = empty(wide, dtype=F32) if c["bias"] else None
    return s


# -- the plain forms ------------------------------------------------------------

def _scores(l, score):
    """[T, E] scores in l's precision, 0 for logits of -inf."""
    if score == "sigmoid":
        return 1 / (1 + torch.exp(-l))
    top = l.amax(dim=1, keepdim=True)
    p = torch.exp(l - torch.where(top == -INF, 0, top))
    total = p.sum(dim=1, keepdim=True)
    return p / torch.where(total == 0, 1, total)


def _plain_route(s):
    c, K = s["case"], s["case"]["K"]
    l = s["logits"].double()  # which of two experts is the larger is settled in 64 bits
    score = _scores(l, c["score"])
    T, E = l.shape
    value = l if s["bias"] is None else score + s["bias"].double()
    value = value.masked_fill(l == -INF, -INF)
    if c["groups"] > 1:
        # (without a bias sums of two are sums of scores)
        v = score.masked_fill(l == -INF, -INF) if c["group_score"] == "top2" and s["bias"] is None else value
        v = v.view(T, c["groups"], -1).sort(dim=2, descending=True).values
        best = v[:, :, 0]
        if c["group_score"] == "top2" and v.shape[2] > 1:
            best = best + v[:, :, 1].masked_fill(v[:, :, 1] == -INF, 0)
        order = best.sort(dim=1, descending=True, stable=True).indices
        kept = torch.zeros_like(best, dtype=torch.bool)
        kept.scatter_(1, order[:, :c["topk_groups"]], True)
        value = value.masked_fill(~kept.repeat_interleave(E // c["groups"], dim=1), -INF)
    top, idx = value.sort(dim=1, descending=True, stable=True)
    top, idx = top[:, :K], idx[:, :K]
    w = score.float().gather(1, idx).masked_fill(top == -INF, 0)
    if c["renorm"]:
        total = w.sum(dim=1, keepdim=True)
        w = w / torch.where(total == 0, 1, total)
    return idx.masked_fill(top == -INF, -1), w * c["scale"]


def _plain_route_grad(s):
    c, idx = s["case"], s["topk_idx"]
    l = s["logits"].float()
    on = idx >= 0
    at = idx.clamp_min(0)
    g = (s["d_topk_w"] * c["scale"]).masked_fill(~on, 0)
    score = _scores(l, c["score"])
    chosen = score.gather(1, at).masked_fill(~on, 0)
    if c["renorm"]:
        total = chosen.sum(dim=1, keepdim=True)
        total = torch.where(total == 0, 1, total)
        g = (g - (g * chosen).sum(dim=1, keepdim=True) / total) / total
        g = g.masked_fill(~on, 0)
    d_score = torch.zeros_like(l).scatter_add_(1, at, g)
    if c["score"] == "sigmoid":
        d = d_score * score * (1 - score)
    else:
        d = score * (d_score - (d_score * score).sum(dim=1, keepdim=True))
    return d.to(s["logits"].dtype)


def _act(z, act):
    if act == "relu":
        return z.clamp_min(0)
    if act == "gelu":
        return 0.5 * z * (1 + torch.erf(z * 0.5 ** 0.5))
    if act == "silu":
        return z / (1 + torch.exp(-z))
    if act == "swiglu":
        gate, up = z.chunk(2, dim=1)
        return gate / (1 + torch.exp(-gate)) * up
    return z


def _plain_linear(s):
    c = s["case"]
    z = s["x"].float() @ s["w"].float().T
    if s["bias"] is not None:
        z = z + s["bias"]
    y = _act(z, c["act"])
    if s["residual"] is not None:
        y = y + s["residual"].float()
    y = y.to(_TYPES[c["out"]])
    return (y, z.to(BF16)) if c["keep_z"] else y


def _plain_linear_grad(s):
    c, dz = s["case"], s["dy"].float()
    if c["act"] != "none":
        z = s["z"].float()
        if c["act"] == "relu":
            dz = dz * (z > 0)
        elif c["act"] == "gelu":
            dz = dz * (0.5 * (1 + torch.erf(z * 0.5 ** 0.5))
                       + z * torch.exp(-0.5 * z * z) * (2 * math.pi) ** -0.5)
        elif c["act"] == "silu":
            q = 1 / (1 + torch.exp(-z))
            dz = dz * q * (1 + z * (1 - q))
        else:
            gate, up = z.chunk(2, dim=1)
            q = 1 / (1 + torch.exp(-gate))
            dz = torch.cat([dz * up * q * (1 + gate * (1 - q)), dz * gate * q], dim=1)
    dx = (dz @ s["w"].float()).to(BF16)
    d_w = (dz.T @ s["x"].float()).to(BF16)
    return (dx, d_w, dz.sum(dim=0)) if c["bias"] else (dx, d_w)


def _plain(s):
    return {"route": _plain_route, "route_grad": _plain_route_grad, "linear": _plain_linear,
            "linear_grad": _plain_linear_grad}[s["case"]["op"]](s)


# -- the framework's operators ----------------------------------------------------

def _own(s):
    from combine_movement_gb300 import ep
    c = s["case"]
    if c["op"] == "route":
        ep.ep_route(s["logits"], s["topk_idx"], s["topk_w"], s["bias"], score=c["score"],
                    groups=c["groups"], topk_groups=c["topk_groups"],
                    group_score=c["group_score"], renormalize=c["renorm"], scale=c["scale"])
        return s["topk_idx"], s["topk_w"]
    if c["op"] == "route_grad":
        ep.ep_route_grad(s["d_topk_w"], s["logits"], s["topk_idx"], s["d_logits"],
                         score=c["score"], renormalize=c["renorm"], scale=c["scale"])
        return s["d_logits"]
    if c["op"] == "linear":
        ep.ep_linear(s["x"], s["w"], s["y"], s["bias"], activation=c["act"],
                     residual=s["residual"], z=s["z"])
        return (s["y"], s["z"]) if c["keep_z"] else s["y"]
    dz = s["dy"]
    if c["act"] != "none" or c["bias"] or c["dy"] != "bf16" or dz.shape[1] % 8:
        dz = s["dz"]
        ep.ep_linear_act_grad(s["dy"], s["z"], dz, s["d_bias"], activation=c["act"])
    ep.ep_linear_grad_input(dz, s["w"], s["dx"])
    ep.ep_linear_grad_weight(dz, s["x"], s["d_w"])
    return (s["dx"], s["d_w"], s["d_bias"]) if c["bias"] else (s["dx"], s["d_w"])


def run(state):
    return _own(state) if own else _plain(state)


# -- floors ------------------------------------------------------------------------

def work(case):
    """Bytes read and written once and operations of one pass."""
    c, T = case, case["T"]
    if c["op"] == "route":
        size = 4 if c["type"] == "f32" else 2
        return {"bytes": size * T * c["E"] + 12 * T * c["K"], "flops": 8 * T * c["E"]}
    if c["op"] == "route_grad":
        size = 4 if c["type"] == "f32" else 2
        dense = c["score"] == "softmax" and not c["renorm"]
        read = c["E"] if dense else c["K"]
        return {"bytes": size * T * (c["E"] + read) + 12 * T * c["K"],
                "flops": (8 * T * c["E"] if dense else 12 * T * c["K"])}
    H, N = c["H"], c["N"]
    wide = 2 * N if c["act"] == "swiglu" else N
    if c["op"] == "linear":
        out = (4 if c["out"] == "f32" else 2) * T * N * (2 if c["residual"] else 1)
        return {"bytes": 2 * T * H + 2 * wide * H + out + (2 * T * wide if c["keep_z"] else 0),
                "flops": 2 * T * H * wide}
    read = (4 if c["dy"] == "f32" else 2) * T * N + (2 * T * wide if c["act"] != "none" else 0)
    return {"bytes": read + 4 * T * H + 4 * wide * H, "flops": 4 * T * H * wide}


# -- 64 bits -------------------------------------------------------------------------

def _exact_chosen(v, K):
    """Indices of the K largest of each row, the first of equal ones; -1 where
    only -inf is left."""
    v, n = v.clone(), torch.arange(v.shape[1], device=v.device)
    out = []
    for _ in range(K):
        top = v.amax(dim=1, keepdim=True)
        at = torch.where(v == top, n, v.shape[1]).amin(dim=1, keepdim=True)
        out.append(torch.where(top == -INF, -1, at))
        v.scatter_(1, at, -INF)
    return torch.cat(out, dim=1)


def _exact_score(l, score):
    return torch.sigmoid(l) if score == "sigmoid" else torch.softmax(l, dim=1).nan_to_num(0.0)


def _exact_route(c, s):
    l = s["logits"].to(F64)
    score = _exact_score(l, c["score"])
    off = l == -INF
    rank = (l if s["bias"] is None else score + s["bias"].to(F64)).masked_fill(off, -INF)
    if c["groups"] > 1:
        size, best = c["E"] // c["groups"], []
        for i in range(0, c["E"], size):
            part = rank[:, i:i + size]
            if c["group_score"] == "max":
                best.append(part.amax(dim=1))
                continue
            two = _exact_chosen(part, min(2, size))
            v = part if s["bias"] is not None else score[:, i:i + size]
            v = torch.where(two < 0, 0.0, v.gather(1, two.clamp_min(0))).sum(dim=1)
            best.append(torch.where(two[:, 0] < 0, -INF, v))
        keep = _exact_chosen(torch.stack(best, dim=1), c["topk_groups"])
        mine = torch.arange(c["E"], device=l.device) // size
        rank = rank.masked_fill((mine[None, :, None] != keep[:, None, :]).all(dim=2), -INF)
    idx = _exact_chosen(rank, c["K"])
    w = torch.where(idx < 0, 0.0, score.gather(1, idx.clamp_min(0)))
    if c["renorm"]:
        w = w / w.sum(dim=1, keepdim=True).clamp_min(1e-300)
    return idx, w * c["scale"]


def _exact_route_grad(c, s):
    # by the chain rule of the definition's own steps
    l = s["logits"].to(F64)
    score, idx = _exact_score(l, c["score"]), s["topk_idx"]
    at, on = idx.clamp_min(0), idx >= 0
    p = torch.where(on, score.gather(1, at), 0.0)
    dw = torch.where(on, s["d_topk_w"].to(F64), 0.0) * c["scale"]
    if c["renorm"]:
        total = p.sum(dim=1, keepdim=True).clamp_min(1e-300)
        dw = torch.where(on, dw / total - (dw * p).sum(dim=1, keepdim=True) / total ** 2, 0.0)
    d = torch.zeros_like(l)
    for k in range(c["K"]):
        d.scatter_add_(1, at[:, k:k + 1], dw[:, k:k + 1])
    if c["score"] == "sigmoid":
        return d * score * torch.sigmoid(-l)
    return score * d - score * (score * d).sum(dim=1, keepdim=True)


def exact(case, seed):
    c, s = case, prepare(case, seed)
    if c["op"] == "route":
        return _exact_route(c, s)
    if c["op"] == "route_grad":
        return _exact_route_grad(c, s)
    x, w = s["x"].to(F64), s["w"].to(F64)
    normal = torch.distributions.Normal(0.0, 1.0)
    if c["op"] == "linear":
        z = torch.mm(x, w.t())
        if s["bias"] is not None:
            z += s["bias"].to(F64)
        y = z
        if c["act"] == "relu":
            y = torch.where(z > 0, z, 0.0)
        elif c["act"] == "gelu":
            y = z * normal.cdf(z)
        elif c["act"] == "silu":
            y = z * torch.sigmoid(z)
        elif c["act"] == "swiglu":
            y = z[:, :c["N"]] * torch.sigmoid(z[:, :c["N"]]) * z[:, c["N"]:]
        if s["residual"] is not None:
            y = y + s["residual"].to(F64)
        return (y, z) if c["keep_z"] else y
    dy = s["dy"].to(F64)
    if c["act"] == "none":
        dz = dy
    else:
        z = s["z"].to(F64)
        a, u = z[:, :c["N"]], z[:, c["N"]:]
        q = torch.sigmoid(a)
        if c["act"] == "relu":
            dz = torch.where(a > 0, dy, 0.0)
        elif c["act"] == "gelu":
            dz = dy * (normal.cdf(a) + a * normal.log_prob(a).exp())
        else:
            slope = q + a * q * torch.sigmoid(-a)
            dz = dy * slope if c["act"] == "silu" else torch.cat([dy * u * slope, dy * a * q], dim=1)
    out = (torch.mm(dz, w), torch.mm(dz.t(), x))
    return out + (dz.sum(dim=0),) if c["bias"] else out
