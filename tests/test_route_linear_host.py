"""Argument checks of the router's and the dense products' calls: each returns
before any CUDA call, so they run without a GPU (addresses are made up and never
used). And the binding's own checks of shapes, types and names."""
import pytest
import torch

A = 0x10000  # a 16-byte aligned address


@pytest.fixture(scope="module")
def ep():
    from combine_movement_gb300 import build
    build.build()
    from combine_movement_gb300 import ep as mod
    return mod


def route(ep, l=A, kind=1, T=8, E=64, K=4, bias=None, score=0, groups=1, kept=1, worth=0, renorm=1,
          scale=1.0, idx=A, w=A):
    return ep.lib.ep_route(l, kind, T, E, K, bias, score, groups, kept, worth, renorm, scale, idx, w,
                           None)


def route_grad(ep, dw=A, l=A, kind=1, idx=A, T=8, E=64, K=4, score=0, renorm=1, scale=1.0, d=A,
               st=None):
    return ep.lib.ep_route_grad(dw, l, kind, idx, T, E, K, score, renorm, scale, d, st, None)


def linear(ep, x=A, M=8, K=64, w=A, N=32, bias=None, act=0, res=None, kind=0, y=A, z=None, st=None):
    return ep.lib.ep_linear(x, M, K, w, N, bias, act, res, kind, y, z, st, None)


def act_grad(ep, dy=A, kind=0, z=A, M=8, N=32, act=3, dz=A, pitch=32, db=None):
    return ep.lib.ep_linear_act_grad(dy, kind, z, M, N, act, dz, pitch, db, None)


def grad_input(ep, dz=A, pitch=32, M=8, N=32, w=A, K=64, dx=A, st=None):
    return ep.lib.ep_linear_grad_input(dz, pitch, M, N, w, K, dx, st, None)


def grad_weight(ep, dz=A, pitch=32, M=8, N=32, x=A, K=64, kind=0, dw=A, acc=0, st=None):
    return ep.lib.ep_linear_grad_weight(dz, pitch, M, N, x, K, kind, dw, acc, st, None)


@pytest.mark.parametrize("call,bad", [
    (route, dict(l=None)), (route, dict(idx=None)), (route, dict(w=None)), (route, dict(l=A + 2)),
    (route, dict(kind=0, l=A + 1)), (route, dict(idx=A + 4)), (route, dict(w=A + 2)),
    (route, dict(bias=A + 1)), (route, dict(kind=2)), (route, dict(kind=-1)), (route, dict(score=2)),
    (route, dict(T=-1)), (route, dict(E=0)), (route, dict(K=0)), (route, dict(K=33)),
    (route, dict(K=65)), (route, dict(E=3, K=4)), (route, dict(groups=0)),
    (route, dict(groups=3, kept=1)), (route, dict(groups=8, kept=0)), (route, dict(groups=8, kept=9)),
    (route, dict(groups=32, kept=1)), (route, dict(worth=2)), (route, dict(groups=-8)),
    (route_grad, dict(dw=None)), (route_grad, dict(l=None)), (route_grad, dict(idx=None)),
    (route_grad, dict(d=None)), (route_grad, dict(d=A + 2)), (route_grad, dict(st=A + 2)),
    (route_grad, dict(kind=5)), (route_grad, dict(score=-1)), (route_grad, dict(K=0)),
    (route_grad, dict(T=-1)), (route_grad, dict(idx=A + 4)),
    (linear, dict(x=None)), (linear, dict(w=None)), (linear, dict(y=None)), (linear, dict(x=A + 8)),
    (linear, dict(w=A + 2)), (linear, dict(y=A + 8)), (linear, dict(res=A + 4)),
    (linear, dict(z=A + 8)), (linear, dict(bias=A + 2)), (linear, dict(st=A + 1)),
    (linear, dict(M=-1)), (linear, dict(N=0)), (linear, dict(K=0)), (linear, dict(K=12)),
    (linear, dict(act=5)), (linear, dict(act=-1)), (linear, dict(kind=2)),
    (act_grad, dict(dy=None)), (act_grad, dict(z=None)), (act_grad, dict(dz=None)),
    (act_grad, dict(pitch=24)), (act_grad, dict(pitch=36)), (act_grad, dict(act=4)),
    (act_grad, dict(act=9)), (act_grad, dict(kind=3)), (act_grad, dict(dy=A + 8)),
    (act_grad, dict(db=A + 1)), (act_grad, dict(M=-2)), (act_grad, dict(N=0)),
    (grad_input, dict(dz=None)), (grad_input, dict(w=None)), (grad_input, dict(dx=None)),
    (grad_input, dict(pitch=24)), (grad_input, dict(N=33, pitch=33)), (grad_input, dict(K=4)),
    (grad_input, dict(dz=A + 8)), (grad_input, dict(dx=A + 2)), (grad_input, dict(st=A + 3)),
    (grad_weight, dict(dz=None)), (grad_weight, dict(x=None)), (grad_weight, dict(dw=None)),
    (grad_weight, dict(M=0, dw=None)), (grad_weight, dict(pitch=16)), (grad_weight, dict(K=20)),
    (grad_weight, dict(kind=4)), (grad_weight, dict(dw=A + 8)), (grad_weight, dict(M=-1)),
])
def test_invalid_arguments(ep, call, bad):
    assert call(ep, **bad) == ep.EP_ERR_INVALID


@pytest.mark.parametrize("call,big", [
    (route, dict(E=4097)), (route, dict(T=1 << 31)), (route, dict(T=1 << 62)),
    (route, dict(groups=64, kept=8)), (route_grad, dict(E=5000)), (route_grad, dict(T=1 << 60)),
    (linear, dict(M=1 << 31)), (linear, dict(N=1 << 31)), (linear, dict(K=1 << 31)),
    (linear, dict(N=1 << 30, act=4)), (linear, dict(M=(1 << 31) - 300, N=1 << 20)),
    (linear, dict(K=1 << 62)), (act_grad, dict(N=1 << 31, pitch=1 << 31)),
    (act_grad, dict(pitch=1 << 31)), (act_grad, dict(M=1 << 31)),
    (grad_input, dict(M=1 << 31)), (grad_input, dict(pitch=1 << 31)),
    (grad_input, dict(M=(1 << 31) - 300, K=1 << 20)), (grad_weight, dict(K=1 << 40)),
    (grad_weight, dict(N=1 << 31, pitch=1 << 31)),
])
def test_sizes_beyond_the_limits(ep, call, big):
    assert call(ep, **big) == ep.EP_ERR_UNSUPPORTED


@pytest.mark.parametrize("call,none", [
    (route, dict(T=0, l=None, idx=None, w=None)), (route_grad, dict(T=0, l=None, idx=None, dw=None)),
    (linear, dict(M=0, x=None, y=None)), (act_grad, dict(M=0, dy=None, z=None)),
    (grad_input, dict(M=0, dz=None, dx=None)), (grad_weight, dict(M=0, dz=None, x=None, acc=1)),
])
def test_nothing_to_do(ep, call, none):
    assert call(ep, **none) == ep.EP_OK


bf, f32, i64 = torch.bfloat16, torch.float32, torch.int64


def z(*shape, dtype=bf):
    return torch.zeros(shape, dtype=dtype)


BINDING = [
    (lambda ep: ep.ep_route(z(4, 8, dtype=torch.float16), z(4, 2, dtype=i64), z(4, 2, dtype=f32)), "logits"),
    (lambda ep: ep.ep_route(z(8, 4).t(), z(4, 2, dtype=i64), z(4, 2, dtype=f32)), "logits.*contiguous"),
    (lambda ep: ep.ep_route(z(8), z(4, 2, dtype=i64), z(4, 2, dtype=f32)), "two dimensions"),
    (lambda ep: ep.ep_route(z(4, 8), z(3, 2, dtype=i64), z(4, 2, dtype=f32)), "topk_idx"),
    (lambda ep: ep.ep_route(z(4, 8), z(4, 2, dtype=torch.int32), z(4, 2, dtype=f32)), "topk_idx"),
    (lambda ep: ep.ep_route(z(4, 8), z(4, 2, dtype=i64), z(4, 2)), "topk_w"),
    (lambda ep: ep.ep_route(z(4, 8), z(4, 2, dtype=i64), z(4, 2, dtype=f32), z(7, dtype=f32)), "bias"),
    (lambda ep: ep.ep_route(z(4, 8), z(4, 2, dtype=i64), z(4, 2, dtype=f32), score="tanh"), "score"),
    (lambda ep: ep.ep_route(z(4, 8), z(4, 2, dtype=i64), z(4, 2, dtype=f32), group_score="sum"), "group_score"),
    (lambda ep: ep.ep_route(z(4, 8), z(4, 2, dtype=i64), z(4, 2, dtype=f32)), "CUDA"),
    (lambda ep: ep.ep_route_grad(z(4, 2, dtype=f32), z(4, 8), z(4, 2, dtype=i64), z(4, 8, dtype=f32)), "d_logits"),
    (lambda ep: ep.ep_route_grad(z(4, 3, dtype=f32), z(4, 8), z(4, 2, dtype=i64), z(4, 8)), "d_topk_w"),
    (lambda ep: ep.ep_route_grad(z(4, 2, dtype=f32), z(4, 8), z(4, 2, dtype=i64), z(4, 8)), "CUDA"),
    (lambda ep: ep.ep_linear(z(4, 8), z(6, 16), z(4, 6)), "w:"),
    (lambda ep: ep.ep_linear(z(4, 8, dtype=f32), z(6, 8), z(4, 6)), "x:"),
    (lambda ep: ep.ep_linear(z(4, 8), z(6, 8), z(4, 5)), "y:"),
    (lambda ep: ep.ep_linear(z(4, 8), z(6, 8), z(4, 6, dtype=torch.float16)), "y:"),
    (lambda ep: ep.ep_linear(z(4, 8), z(8, 6).t(), z(4, 6)), "w:"),
    (lambda ep: ep.ep_linear(z(4, 8), z(7, 8), z(4, 3), activation="swiglu"), "gate half"),
    (lambda ep: ep.ep_linear(z(4, 8), z(6, 8), z(4, 6), activation="tanh"), "activation"),
    (lambda ep: ep.ep_linear(z(4, 8), z(6, 8), z(4, 6), z(6)), "bias"),
    (lambda ep: ep.ep_linear(z(4, 8), z(6, 8), z(4, 6), residual=z(4, 6, dtype=f32)), "residual"),
    (lambda ep: ep.ep_linear(z(4, 8), z(6, 8), z(4, 3), z=z(4, 3), activation="swiglu"), "z:"),
    (lambda ep: ep.ep_linear(z(4, 8), z(6, 8), z(4, 6)), "CUDA"),
    (lambda ep: ep.ep_linear_act_grad(z(4, 6), None, z(4, 8), activation="silu"), "z:"),
    (lambda ep: ep.ep_linear_act_grad(z(4, 6), z(4, 6), z(4, 6), activation="silu"), "dz:"),
    (lambda ep: ep.ep_linear_act_grad(z(4, 6), z(4, 12), z(4, 8), activation="swiglu"), "dz:"),
    (lambda ep: ep.ep_linear_act_grad(z(4, 6), None, z(4, 8), z(5, dtype=f32)), "d_bias"),
    (lambda ep: ep.ep_linear_act_grad(z(4, 6), None, z(4, 8)), "CUDA"),
    (lambda ep: ep.ep_linear_grad_input(z(4, 6), z(6, 8), z(4, 8)), "dz:"),
    (lambda ep: ep.ep_linear_grad_input(z(4, 8), z(6, 8), z(4, 16)), "dx:"),
    (lambda ep: ep.ep_linear_grad_input(z(4, 8), z(6, 8), z(4, 8)), "CUDA"),
    (lambda ep: ep.ep_linear_grad_weight(z(4, 8), z(3, 16), z(6, 16)), "x:"),
    (lambda ep: ep.ep_linear_grad_weight(z(4, 8), z(4, 16), z(6, 16, dtype=torch.float16)), "d_w:"),
    (lambda ep: ep.ep_linear_grad_weight(z(4, 8), z(4, 16), z(6, 16)), "CUDA"),
]


@pytest.mark.parametrize("i", range(len(BINDING)))
def test_binding_refuses(ep, i):
    call, what = BINDING[i]
    with pytest.raises(ValueError, match=what):
        call(ep)


def test_differentiable_calls_refuse(ep):
    from combine_movement_gb300 import moe
    with pytest.raises(ValueError, match="logits"):
        moe.route(z(2, 4, 8), 2)
    with pytest.raises(ValueError, match="x:"):
        moe.linear(z(2, 4, 8), z(4, 8))
