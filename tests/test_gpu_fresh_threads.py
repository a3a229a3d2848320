"""Calls from threads that have made no CUDA call before, as a server's workers are: the
first thing that such a thread asks of the device is the call itself."""
import threading

import pytest
import torch

from test_gpu_expert_fp8 import operands

pytestmark = pytest.mark.gpu
bf, f32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def ep():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    torch.cuda.set_device(0)
    from combine_movement_gb300 import build
    build.build()
    from combine_movement_gb300 import ep as mod
    return mod


def in_a_thread(call):
    """call(), its first and only one, in a thread of its own; what it raised."""
    raised = []

    def run():
        try:
            call()
        except Exception as e:
            raised.append(e)
    t = threading.Thread(target=run)
    t.start()
    t.join()
    torch.cuda.synchronize()
    return raised


def rand(*shape, seed=0, dtype=bf):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return torch.randn(shape, generator=g, device="cuda").to(dtype)


# Outputs and the stream are the caller's, so that nothing else reaches the device first.
@pytest.mark.parametrize("M,N,K", [(1, 64, 64), (128, 256, 4096), (700, 512, 1024), (3000, 2048, 512)])
def test_products(ep, M, N, K):
    x, w, dz = rand(M, K), rand(N, K, seed=1), rand(M, N, seed=2)
    stream = torch.cuda.current_stream().cuda_stream
    calls = [lambda out: ep.ep_linear(x, w, out, stream=stream),
             lambda out: ep.ep_linear_grad_input(dz, w, out, stream=stream),
             lambda out: ep.ep_linear_grad_weight(dz, x, out, stream=stream)]
    for call, shape in zip(calls, ((M, N), (M, K), (N, K))):
        want, got = (torch.full(shape, float("nan"), dtype=bf, device="cuda") for _ in range(2))
        call(want)
        assert in_a_thread(lambda: call(got)) == []
        assert torch.equal(got, want)


def test_expert_products(ep):
    a, a_scale, offsets, w, w_scale = operands([40, 3, 100], 512, 1024, 1)
    stream = torch.cuda.current_stream().cuda_stream
    want, got = (torch.zeros(143, 512, dtype=bf, device="cuda") for _ in range(2))
    ep.ep_expert_matmul_fp8(a, a_scale, offsets, w, w_scale, want, stream=stream)
    assert in_a_thread(lambda: ep.ep_expert_matmul_fp8(a, a_scale, offsets, w, w_scale, got,
                                                       stream=stream)) == []
    assert torch.equal(got, want)


def test_router_and_movement(ep):
    T, E, K, H = 100, 32, 4, 256
    l, x = rand(T, E, dtype=f32), rand(T, H, seed=3)
    stream = torch.cuda.current_stream().cuda_stream
    idx, w = ep.route(l, K)
    _, _, slot = ep.get_dispatch_layout(idx, E)
    rows = ep.dispatch(x, slot, T * K)
    y = ep.combine(rows, slot, w)
    got = [torch.empty_like(t) for t in (idx, w, rows, y)]
    for call in (lambda: ep.ep_route(l, got[0], got[1], stream=stream),
                 lambda: ep.ep_dispatch(x, slot, got[2], stream=stream),
                 lambda: ep.ep_combine(rows, slot, w, got[3], stream=stream)):
        assert in_a_thread(call) == []
    assert all(torch.equal(a, b) for a, b in zip(got, (idx, w, rows, y)))
