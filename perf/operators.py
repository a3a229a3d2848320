"""Workloads of the expert operators around dispatch and combine.

What is timed here, with the plain form of each operator beside the call a
user makes of it:

* ``dispatch_fp8``  -- dispatch with the rows quantised on the way: each row
  block of 128 values goes out as e4m3 with one fp32 scale;
* ``gate_up``       -- the experts' first product, in 8 bits with a scale for
  each block of 128, its two halves joined as silu(gate) * up and quantised;
* ``matmul``        -- the experts' product alone, bf16 out (the down
  projection);
* ``combine_grad``  -- combine's gradient: of the expert rows and of the
  routing weights;
* ``dispatch_grad`` -- dispatch's gradient: each token sums its rows.

``T`` tokens, ``H`` hidden size, ``E`` experts, ``K`` experts per token, ``I``
expert width, ``masked`` the share of routing entries that are -1. Rows are in
receive order (experts ascending, each expert's rows in (token, k) order); the
receive buffers hold T * K rows, and what lies past the unmasked ones stays
zero.
"""
import math

import torch

own = False

BLOCK = 128
E4M3_MAX = 448.0
AMAX_FLOOR = 1e-30  # smallest block maximum a scale is taken from
F8 = torch.float8_e4m3fn

# The largest draws stay within these: bytes moved and operations of one pass.
MOST_BYTES = 4.5e9
MOST_FLOPS = 7.6e12


def listed():
    return [
        # A decode batch of the DeepSeek-V3-shaped layer sent out in 8 bits:
        # 1024 rows, a few microseconds, latency counts.
        {"name": "dispatch_fp8 decode", "op": "dispatch_fp8", "T": 128, "H": 7168, "E": 256, "K": 8,
         "routing": "uniform", "masked": 0.0},
        # The prefill step of the same layer: 32768 rows.
        {"name": "dispatch_fp8 prefill", "op": "dispatch_fp8", "T": 4096, "H": 7168, "E": 256, "K": 8,
         "routing": "uniform", "masked": 0.0},
        # One new token of one sequence: eight experts with one row each; the
        # time is that of reading their weights.
        {"name": "gate_up one token", "op": "gate_up", "T": 1, "H": 7168, "E": 256, "K": 8, "I": 2048,
         "routing": "uniform", "masked": 0.0},
        # The prefill step: about 128 rows for each of 256 experts, ragged;
        # still bound by the weights.
        {"name": "gate_up prefill", "op": "gate_up", "T": 4096, "H": 7168, "E": 256, "K": 8, "I": 2048,
         "routing": "uniform", "masked": 0.0},
        # The largest point of the size sweep: about 1024 rows an expert,
        # bound by the tensor cores.
        {"name": "gate_up long prefill", "op": "gate_up", "T": 16384, "H": 7168, "E": 128, "K": 8,
         "I": 2048, "routing": "uniform", "masked": 0.0},
        # A decode batch's down projection: nearly every expert has rows, on
        # average four; every weight is read for it.
        {"name": "matmul decode", "op": "matmul", "T": 128, "H": 7168, "E": 256, "K": 8, "I": 2048,
         "routing": "uniform", "masked": 0.0},
        # Skewed routing: hot experts with ten times the mean load.
        {"name": "matmul skewed", "op": "matmul", "T": 8192, "H": 4096, "E": 64, "K": 6, "I": 2048,
         "routing": "zipf", "masked": 0.0},
        # Odd everything: a last block of 48 along the inner axis, columns
        # that fill no tile, masked entries, experts without rows.
        {"name": "matmul odd", "op": "matmul", "T": 333, "H": 1000, "E": 24, "K": 3, "I": 1072,
         "routing": "zipf", "masked": 0.2},
        # The tiny workload's training step.
        {"name": "combine_grad tiny", "op": "combine_grad", "T": 128, "H": 1024, "E": 8, "K": 2,
         "routing": "uniform", "masked": 0.0},
        # A training step of the DeepSeek-V3-shaped layer.
        {"name": "combine_grad prefill", "op": "combine_grad", "T": 4096, "H": 7168, "E": 256, "K": 8,
         "routing": "uniform", "masked": 0.0},
        # An odd number of tokens, a tenth of the entries dropped (capacity).
        {"name": "dispatch_grad masked", "op": "dispatch_grad", "T": 999, "H": 2048, "E": 128, "K": 8,
         "routing": "uniform", "masked": 0.1},
        # The skewed layer's training step.
        {"name": "dispatch_grad skewed", "op": "dispatch_grad", "T": 8192, "H": 4096, "E": 64, "K": 6,
         "routing": "zipf", "masked": 0.0},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    while True:
        op = rng.choice(["dispatch_fp8", "gate_up", "matmul", "combine_grad", "dispatch_grad"])
        E = _log_int(rng, 8, 256)
        c = {"op": op, "T": _log_int(rng, 1, 16384), "H": 16 * (2 * _log_int(rng, 8, 224) - 1), "E": E,
             "K": rng.randint(1, min(8, E)), "routing": rng.choice(["uniform", "zipf"]),
             "masked": rng.choice([0.0, 0.0, 0.1, 0.5])}
        if op == "gate_up":
            c["I"] = 128 * rng.choice([1, 2, 3, 5, 7, 11, 16])
        if op == "matmul":
            c["I"] = 16 * _log_int(rng, 8, 128)
            c["H"] += rng.choice([0, 0, 8])
        w = work(c)
        if 2e6 <= w["bytes"] <= MOST_BYTES and w["flops"] <= MOST_FLOPS:
            return c


# -- inputs -------------------------------------------------------------------

def _routing(c, g):
    """topk_idx int64 [T, K]: K distinct experts a token, then the masked
    entries; uniform, or popularity ~ 1 / rank^1.2 without replacement."""
    keys = torch.rand((c["T"], c["E"]), generator=g, device="cuda")
    if c["routing"] == "zipf":
        rank = torch.arange(1, c["E"] + 1, device="cuda", dtype=torch.float32)
        keys = 1.2 * rank.log() + (-(keys.clamp(1e-30, 1 - 2e-7)).log()).log()
    idx = keys.argsort(dim=1)[:, :c["K"]].contiguous()
    if c["masked"]:
        idx[torch.rand(idx.shape, generator=g, device="cuda") < c["masked"]] = -1
    return idx


def _layout(idx, E):
    """counts (host), offsets int32 [E+1], slot int32 [T, K]."""
    flat = idx.reshape(-1)
    key = torch.where(flat < 0, E, flat)
    order = key.argsort(stable=True)
    place = torch.empty_like(order)
    place[order] = torch.arange(order.numel(), device=order.device)
    slot = torch.where(flat < 0, -1, place).to(torch.int32).view(idx.shape)
    counts = torch.bincount(key, minlength=E + 1)[:E]
    offsets = torch.zeros(E + 1, dtype=torch.int32, device=idx.device)
    offsets[1:] = counts.cumsum(0)
    return counts.tolist(), offsets, slot


def _fp8(shape, g):
    """e4m3 values as a block quantiser leaves them: ~N(0, 109), so that a
    block's largest lies near 448."""
    v = torch.randn(shape, generator=g, device="cuda", dtype=torch.bfloat16)
    return v.mul_(109.0).clamp_(-E4M3_MAX, E4M3_MAX).to(F8)


def _scales(shape, mean, g):
    return torch.randn(shape, generator=g, device="cuda").mul_(0.3).exp_().mul_(mean)


def _blocks(n):
    return -(-n // BLOCK)


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed) * 7919 + 17)
    T, H, E, K = c["T"], c["H"], c["E"], c["K"]
    idx = _routing(c, g)
    counts, offsets, slot = _layout(idx, E)
    R = T * K
    s = {"case": c, "counts": counts, "offsets": offsets, "slot": slot}
    bf = torch.bfloat16

    def randn(*shape):
        return torch.randn(shape, generator=g, device="cuda", dtype=bf)

    if c["op"] == "dispatch_fp8":
        # hidden rows with the spread between tokens and the few large
        # channels that make blocks differ
        x = randn(T, H) * torch.exp(0.5 * randn(T, 1))
        x[:, ::H // 7] *= 12
        s["x"] = x
        s["recv_q"] = torch.zeros((R, H), device="cuda", dtype=F8)
        s["recv_scale"] = torch.zeros((R, _blocks(H)), device="cuda")
    elif c["op"] in ("gate_up", "matmul"):
        n, k = (2 * c["I"], H) if c["op"] == "gate_up" else (H, c["I"])
        s["a"] = _fp8((R, k), g)
        s["a_scale"] = _scales((R, _blocks(k)), 1.0 / 109, g)
        s["w"] = _fp8((E, n, k), g)
        s["w_scale"] = _scales((E, _blocks(n), _blocks(k)), 1.0 / 109 / math.sqrt(k), g)
        if c["op"] == "gate_up":
            s["out_q"] = torch.zeros((R, c["I"]), device="cuda", dtype=F8)
            s["out_scale"] = torch.zeros((R, _blocks(c["I"])), device="cuda")
        else:
            s["out"] = torch.zeros((R, n), device="cuda", dtype=bf)
    else:
        s["topk_w"] = torch.randn((T, K), generator=g, device="cuda").softmax(dim=1)
        s["grad"] = randn(T, H) if c["op"] == "combine_grad" else randn(R, H)
        if c["op"] == "combine_grad":
            s["expert_out"] = randn(R, H)
            s["d_expert_out"] = torch.zeros((R, H), device="cuda", dtype=bf)
            s["d_topk_w"] = torch.zeros((T, K), device="cuda")
        else:
            s["dx"] = torch.zeros((T, H), device="cuda", dtype=bf)
    return s


# -- the plain forms ------------------------------------------------------------

def _quantise(v):
    """fp32 [..., n] -> e4m3 [..., n], fp32 scales [..., ceil(n / 128)]."""
    n = v.shape[-1]
    b = torch.nn.functional.pad(v, (0, -n % BLOCK)).unflatten(-1, (-1, BLOCK))
    amax = b.abs().amax(dim=-1, keepdim=True).clamp_min(AMAX_FLOOR)
    top = torch.full_like(amax, E4M3_MAX)
    q = (b * (top / amax)).flatten(-2)[..., :n].to(F8)
    return q, (amax / top).squeeze(-1)


def _plain_product(s):
    """fp32 [R, n]: each expert's rows times its weights, both dequantised;
    zeros past the last expert's rows."""
    live = [e for e, m in enumerate(s["counts"]) if m]
    w, ws = s["w"], s["w_scale"]
    if len(live) < len(s["counts"]):
        at = torch.tensor(live, dtype=torch.long, device=w.device)
        w, ws = w.view(torch.uint8)[at].view(F8), ws[at]
    n, k = w.shape[1:]
    w = w.float()
    w *= ws.repeat_interleave(BLOCK, dim=1)[:, :n].repeat_interleave(BLOCK, dim=2)[:, :, :k]
    a = s["a"].float()
    a *= s["a_scale"].repeat_interleave(BLOCK, dim=1)[:, :k]
    rest = a.shape[0] - sum(s["counts"])
    parts = a.split([s["counts"][e] for e in live] + [rest])[:-1]
    # one product for each expert with rows: they differ in length
    return torch.cat([p @ w[i].T for i, p in enumerate(parts)] + [a.new_zeros((rest, n))])


def _plain(s):
    op = s["case"]["op"]
    if op == "dispatch_fp8":
        q, scale = _quantise(s["x"].float())
        (R, H), slot = s["recv_q"].shape, s["slot"].reshape(-1)
        at = torch.where(slot < 0, R, slot).long()  # masked entries into a row past the end
        token = torch.arange(slot.numel(), device=slot.device) // s["case"]["K"]
        out_q = torch.zeros((R + 1, H), dtype=torch.uint8, device=slot.device)
        out_q[at] = q.view(torch.uint8)[token]
        out_s = scale.new_zeros((R + 1, scale.shape[1]))
        out_s[at] = scale[token]
        return out_q[:R].view(F8), out_s[:R]
    if op == "gate_up":
        gate, up = _plain_product(s).chunk(2, dim=1)
        q, scale = _quantise(gate / (1 + torch.exp(-gate)) * up)
        on = torch.arange(scale.shape[0], device=scale.device)[:, None] < s["offsets"][-1]
        return q, scale * on
    if op == "matmul":
        return _plain_product(s).to(torch.bfloat16)
    slot = s["slot"]
    if op == "dispatch_grad":
        rows = torch.nn.functional.pad(s["grad"], (0, 0, 0, 1))  # masked entries read a zero row
        at = torch.where(slot < 0, rows.shape[0] - 1, slot).long()
        return rows[at].float().sum(dim=1).to(torch.bfloat16)
    rows = torch.nn.functional.pad(s["expert_out"], (0, 0, 0, 1))
    at = torch.where(slot < 0, rows.shape[0] - 1, slot).long()
    dy = s["grad"].float()
    d_w = (rows[at].float() * dy[:, None]).sum(dim=2)
    d_rows = torch.zeros_like(rows)
    d_rows[at] = (dy[:, None] * s["topk_w"][..., None]).to(torch.bfloat16)
    return d_rows[:-1], d_w


# -- the framework's operators ----------------------------------------------------

def _own(s):
    from combine_movement_gb300 import ep
    op = s["case"]["op"]
    if op == "dispatch_fp8":
        ep.ep_dispatch_fp8(s["x"], s["slot"], s["recv_q"], s["recv_scale"])
        return s["recv_q"], s["recv_scale"]
    if op == "gate_up":
        ep.ep_expert_gate_up_fp8(s["a"], s["a_scale"], s["offsets"], s["w"], s["w_scale"],
                                 s["out_q"], s["out_scale"])
        return s["out_q"], s["out_scale"]
    if op == "matmul":
        ep.ep_expert_matmul_fp8(s["a"], s["a_scale"], s["offsets"], s["w"], s["w_scale"], s["out"])
        return s["out"]
    if op == "combine_grad":
        ep.ep_combine_grad(s["grad"], s["expert_out"], s["slot"], s["topk_w"], s["d_expert_out"],
                           s["d_topk_w"])
        return s["d_expert_out"], s["d_topk_w"]
    ep.ep_dispatch_grad(s["grad"], s["slot"], s["dx"])
    return s["dx"]


def run(state):
    return _own(state) if own else _plain(state)


# -- floors ------------------------------------------------------------------------

def work(case):
    """Bytes read and written once and operations of one pass. Rows: the
    unmasked entries; weights: of the experts expected to have rows."""
    c = case
    T, H, E, K = c["T"], c["H"], c["E"], c["K"]
    rows = T * K * (1 - c["masked"])
    if c["op"] == "dispatch_fp8":
        return {"bytes": 2 * T * H + 4 * T * K + rows * (H + 4 * _blocks(H)), "flops": 3 * T * H}
    if c["op"] == "combine_grad":
        return {"bytes": 2 * T * H + 4 * rows * H + 12 * T * K, "flops": 3 * rows * H}
    if c["op"] == "dispatch_grad":
        return {"bytes": 2 * T * H + 2 * rows * H + 4 * T * K, "flops": rows * H}
    share = K * (1 - c["masked"]) / E
    live = E * (1 - (1 - share) ** T)
    if c["routing"] == "zipf":
        p = [(e + 1) ** -1.2 for e in range(E)]
        live = sum(1 - (1 - min(1.0, q / sum(p) * K * (1 - c["masked"]))) ** T for q in p)
    n, k = (2 * c["I"], H) if c["op"] == "gate_up" else (H, c["I"])
    out = rows * (c["I"] + 4 * _blocks(c["I"])) if c["op"] == "gate_up" else 2 * rows * n
    weights = live * (n * k + 4 * _blocks(n) * _blocks(k))
    return {"bytes": weights + rows * (k + 4 * _blocks(k)) + out + 4 * (E + 1),
            "flops": 2 * rows * n * k}


# -- 64 bits -------------------------------------------------------------------------

def _exact_rows(v):
    """Block-quantised rows in 64 bits: (e4m3 values, scales)."""
    q, scales = [], []
    for b in v.split(BLOCK, dim=1):
        amax = torch.clamp(b.abs().max(dim=1, keepdim=True).values, min=AMAX_FLOOR)
        q.append((b / amax * E4M3_MAX).to(F8))
        scales.append(amax / E4M3_MAX)
    return torch.cat([x.double() for x in q], 1), torch.cat(scales, 1)


def exact(case, seed):
    c, s = case, prepare(case, seed)
    op, f64 = c["op"], torch.float64
    slot = s["slot"]
    if op in ("gate_up", "matmul"):
        w, n = s["w"], s["w"].shape[1]
        outs, r0 = [], 0
        for e, m in enumerate(s["counts"]):
            if not m:
                continue
            y = torch.zeros((m, n), dtype=f64, device=w.device)
            for j in range(0, w.shape[2], BLOCK):  # the definition, block by block
                part = s["a"][r0:r0 + m, j:j + BLOCK].to(f64) @ w[e, :, j:j + BLOCK].to(f64).T
                sw = s["w_scale"][e, :, j // BLOCK].to(f64).repeat_interleave(BLOCK)[:n]
                y += part * s["a_scale"][r0:r0 + m, j // BLOCK, None].to(f64) * sw
            outs.append(y)
            r0 += m
        y = torch.cat(outs + [torch.zeros((s["a"].shape[0] - r0, n), dtype=f64, device=w.device)])
        if op == "matmul":
            return y
        gate, up = y[:, :c["I"]], y[:, c["I"]:]
        q, scales = _exact_rows(gate * torch.sigmoid(gate) * up)
        scales[r0:] = 0
        return q, scales
    if op == "dispatch_fp8":
        q, scales = _exact_rows(s["x"].to(f64))
        out_q = torch.zeros(s["recv_q"].shape, dtype=f64, device=q.device)
        out_s = torch.zeros(s["recv_scale"].shape, dtype=f64, device=q.device)
        for k in range(c["K"]):
            t = (slot[:, k] >= 0).nonzero()[:, 0]
            out_q[slot[t, k].long()], out_s[slot[t, k].long()] = q[t], scales[t]
        return out_q, out_s
    if op == "dispatch_grad":
        dx = torch.zeros(s["dx"].shape, dtype=f64, device=slot.device)
        for k in range(c["K"]):
            t = (slot[:, k] >= 0).nonzero()[:, 0]
            dx[t] += s["grad"][slot[t, k].long()].to(f64)
        return dx
    d_rows = torch.zeros(s["d_expert_out"].shape, dtype=f64, device=slot.device)
    d_w = torch.zeros(s["d_topk_w"].shape, dtype=f64, device=slot.device)
    for k in range(c["K"]):
        t = (slot[:, k] >= 0).nonzero()[:, 0]
        r = slot[t, k].long()
        dy = s["grad"][t].to(f64)
        d_rows[r] = dy * s["topk_w"][t, k, None].to(f64)
        d_w[t, k] = (dy * s["expert_out"][r].to(f64)).sum(1)
    return d_rows, d_w
