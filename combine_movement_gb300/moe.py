"""A Mixture-of-Experts layer from the library's calls.

``forward_fp8`` is the layer as it is served, in 8 bits with a scale for each
block of 128 values: layout, quantising dispatch, the experts' gate-up product
with its activation, their down product, combine.

``dispatch`` and ``combine`` are the bf16 movement as differentiable
functions, for training with experts of the caller's own; their backward
passes are ``ep_dispatch_grad`` and ``ep_combine_grad``, and receive rows that
no entry maps to are zero in both directions (``ep_clear_unused_rows``).

``route`` makes the routing table and its weights from a router's logits;
``linear`` is a product in bf16 with bias, activation and residual, for those
logits and for an expert that every token goes through: with h =
linear(x, gate_up, activation="swiglu"), linear(h, down, residual=y) adds it to
combine's y. Both are differentiable. (Like any backward pass, theirs is captured into a
CUDA graph only while no graph of autograd from outside the capture holds the same leaves:
torch would join the two's streams.)

``python -m combine_movement_gb300.moe`` builds a layer with random weights,
runs a batch through it and through a router and a shared expert, compares some
tokens with the layer in fp32 and prints the time of each call as one JSON line.
"""
from __future__ import annotations

from typing import Optional, Tuple

import torch
from torch.autograd import forward_ad

from . import ep


def quantize_weights(w: torch.Tensor) -> Tuple[torch.Tensor, torch.Tensor]:
    """e4m3 [E, N, K] and fp32 scales [E, ceil(N/128), ceil(K/128)] of weights
    [E, N, K], one scale for each block of 128 x 128 (value = e4m3 * scale);
    done once, when the weights are loaded. For a gate-up weight N is 2I, the
    gate half first, I a multiple of 128."""
    b = ep.FP8_BLOCK
    q = torch.empty(w.shape, dtype=torch.float8_e4m3fn, device=w.device)
    scales = []
    for e in range(w.shape[0]):
        n, k = w.shape[1:]
        v = torch.nn.functional.pad(w[e].float(), (0, -k % b, 0, -n % b))
        v = v.view(v.shape[0] // b, b, v.shape[1] // b, b)
        m = v.abs().amax(dim=(1, 3)).clamp_min(1e-30)
        s = m / 448.0
        q[e] = (v / s[:, None, :, None]).clamp(-448, 448).reshape(
            v.shape[0] * b, v.shape[2] * b)[:n, :k].to(torch.float8_e4m3fn)
        scales.append(s)
    return q, torch.stack(scales)


# The movement's calls take their sizes from one tensor; the others' are checked
# here, before anything reads past one.
def _check_shape(t: torch.Tensor, shape: Tuple[int, ...], what: str) -> None:
    if t.shape != shape:
        raise ValueError(f"{what}: expected shape {shape}, got {tuple(t.shape)}")


# Whether one of them carries a forward-mode tangent. No call here has a forward-mode
# derivative: a function of autograd that gets such a tensor says so, the library's
# calls would drop the tangent without a word. (no_grad does not switch it off.)
def _has_tangent(*tensors: Optional[torch.Tensor]) -> bool:
    if getattr(forward_ad, "_current_level", 0) < 0:  # (to ask a tensor takes 0.5 us)
        return False
    return any(t is not None and forward_ad.unpack_dual(t).tangent is not None for t in tensors)


def forward_fp8(x: torch.Tensor, topk_idx: torch.Tensor, topk_w: torch.Tensor,
                w_gate_up: torch.Tensor, s_gate_up: torch.Tensor, w_down: torch.Tensor,
                s_down: torch.Tensor, status: Optional[torch.Tensor] = None) -> torch.Tensor:
    """y[t] = sum over k of topk_w[t,k] * expert_{topk_idx[t,k]}(x[t]), where an
    expert is down(silu(gate(x)) * up(x)).

    x bf16 [T, H], topk_idx int64 [T, K] (-1: unused), topk_w fp32 [T, K];
    w_gate_up e4m3 [E, 2I, H] and w_down e4m3 [E, H, I] with their scales, as
    ``quantize_weights`` makes them. Everything is enqueued on the current
    stream; nothing waits for the device. There is no gradient: where an input
    asks for one, a backward pass through the result raises, and a tangent of
    forward mode is refused."""
    args = (x, topk_idx, topk_w, w_gate_up, s_gate_up, w_down, s_down, status)
    recorded = torch.is_grad_enabled() and any(t is not None and t.requires_grad for t in args)
    if recorded or _has_tangent(*args):
        return _ForwardFp8.apply(*args)
    return _forward_fp8(*args)


def _forward_fp8(x, topk_idx, topk_w, w_gate_up, s_gate_up, w_down, s_down, status):
    T, K = topk_idx.shape
    _check_shape(topk_w, (T, K), "topk_w")
    _check_shape(x, (T, x.shape[-1]), "x")
    _, offsets, slot = ep.get_dispatch_layout(topk_idx, w_gate_up.shape[0], status)
    a, a_scale = ep.dispatch_fp8(x, slot, T * K, status=status)
    h, h_scale = ep.expert_gate_up_fp8(a, a_scale, offsets, w_gate_up, s_gate_up, status)
    out = ep.expert_matmul_fp8(h, h_scale, offsets, w_down, s_down, status)
    return ep.combine(out, slot, topk_w, status)


class _ForwardFp8(torch.autograd.Function):
    """The layer in a graph, whose backward says that it has none."""

    @staticmethod
    def forward(ctx, *args):
        return _forward_fp8(*args)

    @staticmethod
    def backward(ctx, dy):
        raise RuntimeError("forward_fp8 has no gradient: train with moe.dispatch, experts of "
                           "your own and moe.combine")


def _dispatch(x, slot, num_recv):
    recv_x = ep.dispatch(x, slot, num_recv)
    # what the experts make of rows no entry maps to meets a zero gradient in
    # their backward, and zero times whatever the memory held (NaN, infinities)
    # is not zero
    ep.ep_clear_unused_rows(recv_x, slot)
    return recv_x


def _combine_grad(dy, expert_out, slot, topk_w, num_recv, need_w):
    """(d_expert_out of num_recv rows, d_topk_w) of combine; None for the one
    that is not needed (num_recv None, need_w False). expert_out may be None
    without need_w."""
    d_rows = None if num_recv is None else dy.new_empty((num_recv, dy.shape[1]))
    d_w = torch.empty_like(topk_w) if need_w else None
    if d_rows is not None or need_w:
        ep.ep_combine_grad(dy, expert_out, slot, topk_w, d_rows, d_w)
    if d_rows is not None:  # rows no entry maps to have no gradient
        ep.ep_clear_unused_rows(d_rows, slot)
    return d_rows, d_w


# The movement's differentiable functions. Each one's backward is made of the
# others (dispatch is linear, combine bilinear), so that every derivative has
# a graph of its own where one is asked for (create_graph, which leaves the
# gradient mode on in a backward), and refuses a forward-mode tangent.


def _as_function(*grads: Optional[torch.Tensor]) -> bool:
    return torch.is_grad_enabled() or _has_tangent(*grads)


class _Dispatch(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, slot, num_recv):
        ctx.save_for_backward(slot)
        return _dispatch(x, slot, num_recv)

    @staticmethod
    def backward(ctx, d_recv):
        (slot,) = ctx.saved_tensors
        grad = _DispatchGrad.apply if _as_function(d_recv) else ep.dispatch_grad
        return grad(d_recv.contiguous(), slot), None, None


class _DispatchGrad(torch.autograd.Function):
    @staticmethod
    def forward(ctx, d_recv, slot):
        ctx.save_for_backward(slot)
        ctx.num_recv = d_recv.shape[0]
        return ep.dispatch_grad(d_recv, slot)

    @staticmethod
    def backward(ctx, g):
        (slot,) = ctx.saved_tensors
        return _Dispatch.apply(g.contiguous(), slot, ctx.num_recv), None


class _Combine(torch.autograd.Function):
    @staticmethod
    def forward(ctx, expert_out, slot, topk_w):
        # the rows (470 MB at T = 4096, H = 7168, top-8) are for the weights'
        # gradient alone
        rows = expert_out if ctx.needs_input_grad[2] else None
        ctx.save_for_backward(rows, slot, topk_w)
        ctx.num_recv = expert_out.shape[0]
        return ep.combine(expert_out, slot, topk_w)

    @staticmethod
    def backward(ctx, dy):
        expert_out, slot, topk_w = ctx.saved_tensors
        need_rows, _, need_w = ctx.needs_input_grad
        grad = _CombineGrad.apply if _as_function(dy) else _combine_grad
        d_rows, d_w = grad(dy.contiguous(), expert_out, slot, topk_w,
                           ctx.num_recv if need_rows else None, need_w)
        return d_rows, None, d_w


class _CombineGrad(torch.autograd.Function):
    @staticmethod
    def forward(ctx, dy, expert_out, slot, topk_w, num_recv, need_w):
        ctx.set_materialize_grads(False)
        ctx.save_for_backward(dy, expert_out, slot, topk_w)
        return _combine_grad(dy, expert_out, slot, topk_w, num_recv, need_w)

    @staticmethod
    def backward(ctx, g_rows, g_w):
        # d_rows[slot] = w dy and d_w = <dy, expert_out[slot]>, by each factor.
        # dy's two parts are rounded to bf16 before their sum is, as any two
        # gradients of a bf16 tensor that autograd adds.
        dy, expert_out, slot, topk_w = ctx.saved_tensors
        need_dy, need_rows, _, need_w = ctx.needs_input_grad[:4]
        d_dy = d_rows = d_w = None
        if g_rows is not None:
            g_rows = g_rows.contiguous()
            if need_dy:
                d_dy = _Combine.apply(g_rows, slot, topk_w)
            if need_w:
                _, d_w = _CombineGrad.apply(dy, g_rows, slot, topk_w, None, True)
        if g_w is not None:
            g_w = g_w.contiguous()
            if need_dy:
                part = _Combine.apply(expert_out, slot, g_w)
                d_dy = part if d_dy is None else d_dy + part
            if need_rows:
                d_rows, _ = _CombineGrad.apply(dy, None, slot, g_w, expert_out.shape[0], False)
        return d_dy, d_rows, None, d_w, None, None


def dispatch(x: torch.Tensor, slot: torch.Tensor, num_recv: int) -> torch.Tensor:
    """``ep.dispatch`` with a gradient for x, of any order. Rows of the result
    that no entry maps to are zero."""
    _check_shape(slot, (x.shape[0], slot.shape[-1]), "slot")
    return _Dispatch.apply(x.contiguous(), slot, num_recv)


def combine(expert_out: torch.Tensor, slot: torch.Tensor, topk_w: torch.Tensor) -> torch.Tensor:
    """``ep.combine`` with gradients for the expert rows and the weights, of any
    order."""
    _check_shape(slot, (topk_w.shape[0], slot.shape[-1]), "slot")
    _check_shape(topk_w, tuple(slot.shape), "topk_w")
    return _Combine.apply(expert_out.contiguous(), slot, topk_w)


def _refuse_tangent(name: str, t: torch.Tensor) -> None:
    if _has_tangent(t):
        raise NotImplementedError(f"{name}: no forward-mode derivative of its backward pass")


class _Route(torch.autograd.Function):
    @staticmethod
    def forward(ctx, logits, k, bias, kind, status):
        idx, w = ep.route(logits, k, bias, **kind)
        ctx.save_for_backward(logits, idx)
        ctx.kind = dict({n: kind[n] for n in ("score", "renormalize", "scale")}, status=status)
        ctx.mark_non_differentiable(idx)
        return idx, w

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, _, d_w):
        _refuse_tangent("route", d_w)
        logits, idx = ctx.saved_tensors
        return ep.route_grad(d_w.contiguous(), logits, idx, **ctx.kind), None, None, None, None


def route(logits: torch.Tensor, k: int, bias: Optional[torch.Tensor] = None,
          score: str = "softmax", groups: int = 1, topk_groups: int = 1, group_score: str = "max",
          renormalize: bool = True, scale: float = 1.0, status: Optional[torch.Tensor] = None
          ) -> Tuple[torch.Tensor, torch.Tensor]:
    """``ep.route`` -- (topk_idx int64 [T, k], topk_w fp32 [T, k]), what layout and
    combine take -- with a gradient of topk_w for the logits, once (a second
    derivative raises). The bias, for the choice alone, has none. ``status`` is the
    backward pass's."""
    _check_shape(logits, (logits.shape[0], logits.shape[-1]), "logits")
    return _Route.apply(logits.contiguous(), k, None if bias is None else bias.detach(),
                        dict(score=score, groups=groups, topk_groups=topk_groups,
                             group_score=group_score, renormalize=renormalize, scale=scale), status)


# Rows as the products read them: a copy where they do not lie one after the other or
# do not start on 16 bytes (flat parameters, the gradient of one of several results that
# were joined).
def _dense(t: torch.Tensor) -> torch.Tensor:
    t = t.contiguous()
    return t if t.data_ptr() % 16 == 0 else t.clone()


class _Linear(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, w, bias, residual, activation, out_dtype, status):
        M, wide = x.shape[0], w.shape[0]
        y = x.new_empty((M, wide // 2 if activation == "swiglu" else wide), dtype=out_dtype)
        need = any(ctx.needs_input_grad[:3])
        z = x.new_empty((M, wide)) if need and activation != "none" else None
        ep.ep_linear(x, w, y, bias, activation, residual, z, status)
        # the rows are for the weight's gradient alone, the weight for the rows'
        ctx.save_for_backward(x if ctx.needs_input_grad[1] else None,
                              w if ctx.needs_input_grad[0] else None, z)
        ctx.activation, ctx.wide, ctx.status = activation, wide, status
        return y

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dy):
        x, w, z = ctx.saved_tensors
        need_x, need_w, need_bias, need_residual = ctx.needs_input_grad[:4]
        if need_x or need_w or need_bias:
            _refuse_tangent("linear", dy)
        dy, wide, act = _dense(dy), ctx.wide, ctx.activation
        M = dy.shape[0]
        dx = d_w = d_bias = None
        dz = dy  # where it is what the products take
        if act != "none" or dy.dtype is not torch.bfloat16 or wide % 8:
            dz = None
            if need_x or need_w:
                dz = dy.new_empty((M, ep.linear_pitch(wide)), dtype=torch.bfloat16)
        if need_bias:
            d_bias = dy.new_empty(wide, dtype=torch.float32)
        if need_bias or dz is not dy and dz is not None:
            ep.ep_linear_act_grad(dy, z, None if dz is dy else dz, d_bias, act)
        if need_x:
            dx = dz.new_empty((M, w.shape[1]))
            ep.ep_linear_grad_input(dz, w, dx, ctx.status)
        if need_w:
            d_w = dz.new_empty((wide, x.shape[1]))
            ep.ep_linear_grad_weight(dz, x, d_w, status=ctx.status)
        return dx, d_w, d_bias, dy if need_residual else None, None, None, None


def linear(x: torch.Tensor, w: torch.Tensor, bias: Optional[torch.Tensor] = None,
           activation: str = "none", residual: Optional[torch.Tensor] = None,
           out_dtype: torch.dtype = torch.bfloat16, status: Optional[torch.Tensor] = None
           ) -> torch.Tensor:
    """act(x w^T + bias) + residual with gradients for all four, once (a second
    derivative raises): x bf16 [M, K], w bf16 [N, K] (swiglu: [2N, K], the gate
    half first), bias fp32, residual [M, N] of out_dtype, which is bf16 or, for a
    router's logits, fp32. Keeps x w^T + bias in bf16 where an activation's
    gradient wants it, and rounds what comes back, through the activation or in fp32,
    to bf16 before the gradients' products. ``status`` (int32 [1]) takes what a product reports,
    here and in the backward pass: after a wait that gave up results are not whole."""
    _check_shape(x, (x.shape[0], w.shape[-1]), "x")
    x, w, residual = _dense(x), _dense(w), None if residual is None else _dense(residual)
    # (a function's forward is not told that no gradient is recorded, and would keep z)
    if not torch.is_grad_enabled() and not _has_tangent(x, w, bias, residual):
        return ep.linear(x, w, bias, activation, residual, out_dtype, status)
    return _Linear.apply(x, w, bias, residual, activation, out_dtype, status)


def _main() -> None:
    import argparse
    import json

    from . import workloads as W

    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--workload", default="decode", choices=sorted(W.BY_NAME))
    ap.add_argument("--width", type=int, default=2048, help="expert width (a multiple of 128)")
    ap.add_argument("--steps", type=int, default=20)
    args = ap.parse_args()
    inp = W.make_inputs(W.BY_NAME[args.workload])
    wl, dev = inp.wl, torch.device("cuda")
    x, idx, w = inp.x.to(dev), inp.topk_idx.to(dev), inp.topk_w.to(dev)
    g = torch.Generator(device=dev)
    g.manual_seed(wl.seed)

    def weights(n, k):
        """random e4m3 weights, a block's values up to 448"""
        q = torch.randn((wl.E, n, k), generator=g, device=dev, dtype=torch.bfloat16)
        q = q.mul_(109).clamp_(-448, 448).to(torch.float8_e4m3fn)
        return q, torch.full((wl.E, -(-n // 128), -(-k // 128)), k ** -0.5 / 109, device=dev)

    gate_up, down = weights(2 * args.width, wl.H), weights(wl.H, args.width)
    status = torch.zeros(1, dtype=torch.int32, device=dev)
    y = forward_fp8(x, idx, w, *gate_up, *down, status)
    assert ep.ep_get_status(status) == ep.EP_OK

    tokens = range(min(wl.T, 4))
    worst = 0.0
    for t in tokens:
        want = torch.zeros(wl.H, device=dev)
        for k in range(wl.K):
            e = int(idx[t, k])
            gu = (gate_up[0][e].float() * gate_up[1][e, 0, 0]) @ x[t].float()
            h = torch.nn.functional.silu(gu[:args.width]) * gu[args.width:]
            want += w[t, k] * ((down[0][e].float() * down[1][e, 0, 0]) @ h)
        worst = max(worst, float((y[t].float() - want).norm() / want.norm()))

    T, K = idx.shape
    _, offsets, slot = ep.get_dispatch_layout(idx, wl.E)
    a, a_scale = ep.dispatch_fp8(x, slot, T * K)
    h, h_scale = ep.expert_gate_up_fp8(a, a_scale, offsets, *gate_up)
    out = ep.expert_matmul_fp8(h, h_scale, offsets, *down)
    calls = {
        "layout": lambda: ep.get_dispatch_layout(idx, wl.E),
        "dispatch_fp8": lambda: ep.ep_dispatch_fp8(x, slot, a, a_scale),
        "gate_up": lambda: ep.ep_expert_gate_up_fp8(a, a_scale, offsets, *gate_up, h, h_scale),
        "down": lambda: ep.ep_expert_matmul_fp8(h, h_scale, offsets, *down, out),
        "combine": lambda: ep.ep_combine(out, slot, w, y),
        "layer": lambda: forward_fp8(x, idx, w, *gate_up, *down),
    }

    # the router of this layer, and a shared expert of the same width
    def dense(n, k):
        return torch.randn((n, k), generator=g, device=dev, dtype=torch.bfloat16) * k ** -0.5

    gate, s13, s2 = dense(wl.E, wl.H), dense(2 * args.width, wl.H), dense(wl.H, args.width)
    logits = ep.linear(x, gate, out_dtype=torch.float32, status=status)
    own_idx, own_w = ep.route(logits, wl.K, score="sigmoid")
    hidden = ep.linear(x, s13, activation="swiglu", status=status)
    y_all = ep.linear(hidden, s2, residual=y, status=status)
    assert ep.ep_get_status(status) == ep.EP_OK
    assert torch.equal(own_idx, logits.sort(dim=1, descending=True, stable=True).indices[:, :wl.K])
    worst_shared = 0.0
    for t in tokens:
        gu = s13.float() @ x[t].float()
        want = s2.float() @ (torch.nn.functional.silu(gu[:args.width]) * gu[args.width:])
        worst_shared = max(worst_shared, float((y_all[t].float() - y[t].float() - want).norm()
                                               / want.norm()))
    calls.update({
        "router_logits": lambda: ep.ep_linear(x, gate, logits),
        "route": lambda: ep.ep_route(logits, own_idx, own_w, score="sigmoid"),
        "shared_gate_up": lambda: ep.ep_linear(x, s13, hidden, activation="swiglu"),
        "shared_down": lambda: ep.ep_linear(hidden, s2, y_all, residual=y),
    })
    us = {}
    for name, call in calls.items():
        for _ in range(3):
            call()
        begin, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
        begin.record()
        for _ in range(args.steps):
            call()
        end.record()
        end.synchronize()
        us[name] = round(begin.elapsed_time(end) / args.steps * 1e3, 2)
    print(json.dumps({"workload": wl.name, "T": T, "H": wl.H, "E": wl.E, "K": K,
                      "width": args.width, "us": us,
                      "relative_error_against_fp32": round(worst, 4),
                      "shared_relative_error_against_fp32": round(worst_shared, 4)}))


if __name__ == "__main__":
    _main()
