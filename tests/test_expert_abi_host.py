"""Argument checks of the expert and gradient calls: each returns before any
CUDA call, so they run without a GPU (addresses are made up and never used).
And the binding's own checks of shapes and types."""
import pytest
import torch

A = 0x10000  # a 16-byte aligned address


@pytest.fixture(scope="module")
def ep():
    from combine_movement_gb300 import build
    build.build()
    from combine_movement_gb300 import ep as mod
    return mod


def matmul(ep, a=A, s=A, R=8, off=A, E=4, w=A, ws=A, N=256, K=128, out=A, st=None):
    return ep.lib.ep_expert_matmul_fp8(a, s, R, off, E, w, ws, N, K, out, st, None)


def gate_up(ep, a=A, s=A, R=8, off=A, E=4, w=A, ws=A, I=128, K=128, q=A, qs=A, st=None):
    return ep.lib.ep_expert_gate_up_fp8(a, s, R, off, E, w, ws, I, K, q, qs, st, None)


def dispatch(ep, x=A, T=8, H=128, K=2, slot=A, w=None, R=16, q=A, s=A, rw=None, rs=None, st=None):
    return ep.lib.ep_dispatch_fp8(x, T, H, K, slot, w, R, q, s, rw, rs, st, None)


def combine_grad(ep, dy=A, e=A, R=16, slot=A, w=A, T=8, H=128, K=2, de=A, dw=A, st=None):
    return ep.lib.ep_combine_grad(dy, e, R, slot, w, T, H, K, de, dw, st, None)


def dispatch_grad(ep, d=A, R=16, slot=A, T=8, H=128, K=2, dx=A, st=None):
    return ep.lib.ep_dispatch_grad(d, R, slot, T, H, K, dx, st, None)


@pytest.mark.parametrize("call,bad", [
    (matmul, dict(a=None)), (matmul, dict(s=None)), (matmul, dict(off=None)), (matmul, dict(w=None)),
    (matmul, dict(ws=None)), (matmul, dict(out=None)), (matmul, dict(a=A + 8)),
    (matmul, dict(w=A + 8)), (matmul, dict(out=A + 2)), (matmul, dict(s=A + 2)),
    (matmul, dict(off=A + 1)), (matmul, dict(st=A + 2)), (matmul, dict(R=-1)), (matmul, dict(E=0)),
    (matmul, dict(N=0)), (matmul, dict(N=12)), (matmul, dict(K=0)), (matmul, dict(K=24)),
    (gate_up, dict(I=64)), (gate_up, dict(I=0)), (gate_up, dict(I=-128)), (gate_up, dict(K=8)),
    (gate_up, dict(q=None)), (gate_up, dict(qs=None)), (gate_up, dict(q=A + 8)),
    (gate_up, dict(qs=A + 2)), (gate_up, dict(a=None)), (gate_up, dict(R=-3)),
    (dispatch, dict(H=24)), (dispatch, dict(H=0)), (dispatch, dict(T=-1)), (dispatch, dict(K=33)),
    (dispatch, dict(x=None)), (dispatch, dict(slot=None)), (dispatch, dict(q=None)),
    (dispatch, dict(s=None)), (dispatch, dict(q=A + 8)), (dispatch, dict(s=A + 2)),
    (dispatch, dict(rw=A)), (dispatch, dict(x=A + 2)),
    (combine_grad, dict(dy=None)), (combine_grad, dict(e=None)), (combine_grad, dict(slot=None)),
    (combine_grad, dict(w=None)), (combine_grad, dict(de=None, dw=None)),
    (combine_grad, dict(H=12)), (combine_grad, dict(K=0)), (combine_grad, dict(de=A + 8)),
    (combine_grad, dict(dw=A + 2)), (combine_grad, dict(w=A + 2)), (combine_grad, dict(R=-1)),
    (dispatch_grad, dict(d=None)), (dispatch_grad, dict(dx=None)), (dispatch_grad, dict(slot=None)),
    (dispatch_grad, dict(d=A + 4)), (dispatch_grad, dict(H=4)), (dispatch_grad, dict(T=-2)),
])
def test_invalid_arguments(ep, call, bad):
    assert call(ep, **bad) == ep.EP_ERR_INVALID


@pytest.mark.parametrize("call,big", [
    (matmul, dict(E=5000)), (matmul, dict(R=1 << 31)), (matmul, dict(K=1 << 31)),
    (matmul, dict(E=4096, N=1 << 20)), (matmul, dict(N=1 << 62)),
    (matmul, dict(E=1, R=(1 << 31) - 1, N=1 << 16)), (gate_up, dict(E=1, R=(1 << 31) - 1, I=1 << 15)), (matmul, dict(K=1 << 62)),
    (gate_up, dict(I=1 << 40)), (gate_up, dict(I=1 << 30)), (gate_up, dict(E=4097)),
    (dispatch, dict(T=1 << 31)), (dispatch, dict(T=1 << 62)), (dispatch, dict(R=1 << 31)),
    (dispatch, dict(H=1 << 31)),
    (combine_grad, dict(T=1 << 31)), (combine_grad, dict(R=1 << 31)), (combine_grad, dict(H=1 << 40)),
    (dispatch_grad, dict(T=1 << 60)), (dispatch_grad, dict(H=1 << 31)),
])
def test_sizes_beyond_the_limits(ep, call, big):
    assert call(ep, **big) == ep.EP_ERR_UNSUPPORTED


def test_nothing_to_do_needs_no_gpu(ep):
    assert matmul(ep, a=None, s=None, R=0, off=None, w=None, ws=None, out=None) == ep.EP_OK
    assert gate_up(ep, a=None, s=None, R=0, off=None, w=None, ws=None, q=None, qs=None) == ep.EP_OK
    assert dispatch(ep, x=None, T=0, slot=None, q=None, s=None) == ep.EP_OK
    assert combine_grad(ep, dy=None, e=None, slot=None, w=None, T=0, de=None, dw=None) == ep.EP_OK
    assert dispatch_grad(ep, d=None, slot=None, T=0, dx=None) == ep.EP_OK


def test_binding_checks_shapes(ep):
    f8, bf, f32, i32 = torch.float8_e4m3fn, torch.bfloat16, torch.float32, torch.int32
    a, s = torch.zeros((6, 256), dtype=f8), torch.zeros((6, 2), dtype=f32)
    off = torch.zeros(4, dtype=i32)
    w, ws = torch.zeros((3, 256, 256), dtype=f8), torch.zeros((3, 2, 2), dtype=f32)
    out = torch.zeros((6, 256), dtype=bf)
    good = dict(a=a, a_scale=s, offsets=off, w=w, w_scale=ws, out=out)
    for bad in (dict(a_scale=s[:, :1]), dict(offsets=off[:3]), dict(w=w[:, :, :128]),
                dict(w_scale=ws[:, :1]), dict(out=out[:5]), dict(a_scale=s[:5])):
        with pytest.raises(ValueError, match="expected shape"):
            ep.ep_expert_matmul_fp8(**{**good, **bad})
    with pytest.raises(ValueError, match="CUDA tensor"):
        ep.ep_expert_matmul_fp8(**good)
    with pytest.raises(ValueError, match="gate half"):
        ep.ep_expert_gate_up_fp8(a, s, off, w[:, :255], ws, a, s)
    x, slot = torch.zeros((5, 128), dtype=bf), torch.zeros((5, 2), dtype=i32)
    q, qs = torch.zeros((10, 128), dtype=f8), torch.zeros((10, 1), dtype=f32)
    for bad in (dict(slot=slot[:4]), dict(recv_q=q[:, :64]), dict(recv_scale=qs[:9])):
        with pytest.raises(ValueError, match="expected shape"):
            ep.ep_dispatch_fp8(**{**dict(x=x, slot=slot, recv_q=q, recv_scale=qs), **bad})
    e, tw = torch.zeros((10, 128), dtype=bf), torch.zeros((5, 2))
    grads = dict(dy=x, expert_out=e, slot=slot, topk_w=tw, d_expert_out=e, d_topk_w=tw)
    for bad in (dict(expert_out=e[:, :64]), dict(slot=slot[1:]), dict(topk_w=tw[:, :1]),
                dict(d_expert_out=e[:9]), dict(d_topk_w=tw[:4])):
        with pytest.raises(ValueError, match="expected shape"):
            ep.ep_combine_grad(**{**grads, **bad})
    with pytest.raises(ValueError, match="expected shape"):
        ep.ep_dispatch_grad(e[:, :64], slot, x)
    with pytest.raises(ValueError, match="expected shape"):
        ep.ep_dispatch_grad(e, slot[:3], x)
