"""The MoE layer of the library's calls: the 8-bit forward against the layer in
64 bits, and the differentiable movement against torch's own gradients."""
import numpy as np
import pytest
import torch

from combine_movement_gb300 import workloads as W

pytestmark = pytest.mark.gpu
f64 = torch.float64


@pytest.fixture(scope="module")
def mods():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    torch.cuda.set_device(0)
    from combine_movement_gb300 import build
    build.build()
    from combine_movement_gb300 import ep, moe
    return ep, moe


def layer(T, H, E, K, width, seed, mask=0.0):
    wl = W.Workload("layer", T=T, H=H, E=E, K=K, seed=seed, mask_frac=mask)
    inp = W.make_inputs(wl)
    g = torch.Generator().manual_seed(seed)
    gate_up = torch.randn((E, 2 * width, H), generator=g) * H ** -0.5
    down = torch.randn((E, H, width), generator=g) * width ** -0.5
    return (inp.x.cuda(), inp.topk_idx.cuda(), inp.topk_w.cuda(), gate_up.cuda(), down.cuda())


def spread(q, s):
    """fp64 weights that a quantised one stands for."""
    n, k = q.shape[1:]
    s = s.to(f64).repeat_interleave(128, 1)[:, :n].repeat_interleave(128, 2)[:, :, :k]
    return q.to(f64) * s


def exact(x, idx, w, gate_up, down):
    """The layer in 64 bits (of unquantised rows), and the norm of what is summed."""
    y = torch.zeros(x.shape, dtype=f64, device=x.device)
    width = gate_up.shape[1] // 2
    for e in range(gate_up.shape[0]):
        t, k = (idx == e).nonzero(as_tuple=True)
        gu = x[t].to(f64) @ gate_up[e].T
        h = gu[:, :width] * torch.sigmoid(gu[:, :width]) * gu[:, width:]
        y.index_add_(0, t, w[t, k, None].to(f64) * (h @ down[e].T))
    return y


@pytest.mark.parametrize("T,H,E,K,width,mask", [
    (1, 512, 16, 4, 256, 0.0), (130, 1040, 8, 2, 128, 0.0), (257, 512, 24, 3, 384, 0.3),
    (700, 1024, 4, 4, 512, 0.0)])
def test_forward_fp8(mods, T, H, E, K, width, mask):
    """Rounding rows to e4m3 makes each value off by at most 2^-4, on average
    over the mantissas (uniform error of half a step, steps of 2^-3 to 2^-4 of
    the value) by about 0.026 of it in the mean square. Products of many
    independent such errors keep that relative size; it enters once at the
    rows and once at h, through silu(g) u, where both factors carry the rows'
    error: sqrt(2) to 2 times 0.026. Together below
    sqrt((2 * 0.026)^2 + 0.026^2) = 0.058; 0.08 with room for tokens' spread."""
    ep, moe = mods
    x, idx, w, gate_up, down = layer(T, H, E, K, width, seed=T, mask=mask)
    q1, s1 = moe.quantize_weights(gate_up)
    q2, s2 = moe.quantize_weights(down)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    y = moe.forward_fp8(x, idx, w, q1, s1, q2, s2, status)
    assert ep.ep_get_status(status) == ep.EP_OK
    want = exact(x, idx, w, spread(q1, s1), spread(q2, s2))
    assert float((y.to(f64) - want).norm() / want.norm()) < 0.08
    none = (idx < 0).all(1)
    assert bool((y[none] == 0).all())


def test_quantize_weights(mods):
    ep, moe = mods
    w = torch.randn((3, 200, 144), device="cuda") * torch.exp(torch.randn((3, 1, 1), device="cuda"))
    w[1, :128, :128] = 0
    q, s = moe.quantize_weights(w)
    assert q.shape == w.shape and s.shape == (3, 2, 2)
    err = (spread(q, s) - w.to(f64)).abs()
    step = spread(torch.ones_like(q), s)
    assert bool((err <= w.abs().to(f64) * (2.0 ** -4 + 2.0 ** -20) + step * 2.0 ** -10).all())


def test_training_movement(mods):
    """Gradients through dispatch, an expert of torch's and combine against
    the same layer in 64 bits; bf16 rounds each of the four movements and the
    expert's product (relative 2^-8 each, rms half of that): 0.02 of the norm."""
    ep, moe = mods
    T, H, E, K = 120, 256, 6, 3
    x, idx, w, _, _ = layer(T, H, E, K, 128, seed=3, mask=0.2)
    _, offsets, slot = ep.get_dispatch_layout(idx, E)
    g = torch.Generator(device="cuda").manual_seed(1)
    m = (torch.randn((H, H), generator=g, device="cuda") * H ** -0.5).to(torch.bfloat16)
    dy = torch.randn((T, H), generator=g, device="cuda").to(torch.bfloat16)
    x.requires_grad_()
    w.requires_grad_()
    m.requires_grad_()
    R = int(offsets[-1])
    y = moe.combine(moe.dispatch(x, slot, R) @ m, slot, w)
    y.backward(dy)
    x64, w64, m64 = (v.detach().to(f64).requires_grad_() for v in (x, w, m))
    on = (idx >= 0).to(f64)[..., None]
    y64 = (w64[..., None] * on * (x64 @ m64)[:, None]).sum(1)
    y64.backward(dy.to(f64))
    for got, want in ((y, y64), (x.grad, x64.grad), (w.grad, w64.grad), (m.grad, m64.grad)):
        err = (got.detach().to(f64) - want.detach()).norm() / want.detach().norm()
        assert float(err) < 0.02


def test_unused_rows_bring_nothing_into_the_gradients(mods):
    ep, moe = mods
    x, idx, w, _, _ = layer(20, 64, 4, 2, 128, seed=4, mask=0.5)
    _, _, slot = ep.get_dispatch_layout(idx, 4)
    rows = torch.randn((40, 64), device="cuda").to(torch.bfloat16).requires_grad_()
    moe.combine(rows, slot, w).sum().backward()
    used = torch.zeros(40, dtype=torch.bool, device="cuda")
    used[slot[slot >= 0].long()] = True
    assert bool((rows.grad[~used] == 0).all()) and bool((rows.grad[used] != 0).any())


def test_same_bits_on_streams_partitions_and_overlap_modes(mods):
    """The layer on three streams and both streams of an SM partition at once,
    and under each launch-overlap mode: the results of a quiet GPU."""
    ep, moe = mods
    x, idx, w, gate_up, down = layer(300, 512, 16, 4, 256, seed=11, mask=0.1)
    args = (x, idx, w, *moe.quantize_weights(gate_up), *moe.quantize_weights(down))
    want = moe.forward_fp8(*args)
    part, rest, _, _ = ep.ep_sm_partition(24)
    streams = [torch.cuda.Stream() for _ in range(3)]
    streams += [torch.cuda.ExternalStream(part), torch.cuda.ExternalStream(rest)]
    torch.cuda.synchronize()
    for _ in range(10):
        got = []
        for s in streams:
            with torch.cuda.stream(s):
                got.append(moe.forward_fp8(*args))
        torch.cuda.synchronize()
        assert all(torch.equal(y, want) for y in got)
    try:
        for mode in (1, 2):
            ep.ep_set_launch_overlap(mode)
            for _ in range(10):
                assert torch.equal(moe.forward_fp8(*args), want)
    finally:
        ep.ep_set_launch_overlap(0)


def test_command(mods, capsys, monkeypatch):
    import json
    import sys
    ep, moe = mods
    monkeypatch.setattr(sys, "argv", ["moe", "--workload", "tiny", "--width", "256", "--steps", "2"])
    moe._main()
    line = json.loads(capsys.readouterr().out.strip().splitlines()[-1])
    assert line["us"]["layer"] > 0 and line["relative_error_against_fp32"] < 0.08
