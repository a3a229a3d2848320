"""The layer with its router and an expert that every token goes through, as a
training step runs it: logits, route, layout, dispatch, experts, combine, the shared
expert added to the result; forward and gradients against the same layer in 64
bits with the same choice.

Tolerances. Every step rounds its result to bf16 (2^-8 of it); a result's path
has at most 8 of those, and as many again on a gradient's way back, each of
which enters what follows with at most the norm of what it came from: 16 * 2^-8
of the norm is far from what a wrong term would give.
"""
import pytest
import torch

pytestmark = pytest.mark.gpu
f64, bf = torch.float64, torch.bfloat16
F = torch.nn.functional


@pytest.fixture(scope="module")
def mods():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    torch.cuda.set_device(0)
    from combine_movement_gb300 import build
    build.build()
    from combine_movement_gb300 import ep, moe
    return ep, moe


def rand(*shape, seed, scale=1.0, dtype=bf):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda") * scale).to(dtype)


T, H, E, K, I = 200, 256, 24, 4, 136
KIND = dict(score="sigmoid", groups=4, topk_groups=2, group_score="top2", scale=1.5)


def leaves():
    return {"x": rand(T, H, seed=1), "gate": rand(E, H, seed=2, scale=H ** -0.5),
            "w1": rand(E, I, H, seed=3, scale=H ** -0.5), "w2": rand(E, H, I, seed=4, scale=I ** -0.5),
            "s1": rand(2 * I, H, seed=5, scale=H ** -0.5), "s2": rand(H, I, seed=6, scale=I ** -0.5),
            "b2": rand(H, seed=7, scale=0.1, dtype=torch.float32)}


def layer(ep, moe, p, bias):
    logits = moe.linear(p["x"], p["gate"], out_dtype=torch.float32)
    idx, w = moe.route(logits, K, bias, **KIND)
    counts, _, slot = ep.get_dispatch_layout(idx, E)
    rows = moe.dispatch(p["x"], slot, T * K)
    out = torch.cat([moe.linear(moe.linear(r, p["w1"][e], activation="silu"), p["w2"][e])
                     for e, r in enumerate(rows.split(counts.tolist() + [T * K - int(counts.sum())])[:E])])
    out = torch.cat([out, rows.new_zeros(T * K - out.shape[0], H)])
    y = moe.combine(out, slot, w)
    h = moe.linear(p["x"], p["s1"], activation="swiglu")
    return moe.linear(h, p["s2"], p["b2"], residual=y), idx


def layer64(p, idx):
    p = {k: v.to(f64) for k, v in p.items()}
    s = torch.sigmoid(p["x"] @ p["gate"].T).gather(1, idx)
    w = KIND["scale"] * s / s.sum(dim=1, keepdim=True)
    out = torch.stack([F.silu(p["x"] @ p["w1"][e].T) @ p["w2"][e].T for e in range(E)], dim=1)
    y = (w[..., None] * out.gather(1, idx[..., None].expand(-1, -1, H))).sum(dim=1)
    g, u = (p["x"] @ p["s1"].T).chunk(2, dim=1)
    return (F.silu(g) * u) @ p["s2"].T + p["b2"] + y


def run(mods):
    p = {k: v.requires_grad_(True) for k, v in leaves().items()}
    bias = rand(E, seed=8, scale=0.1, dtype=torch.float32)
    y, idx = layer(*mods, p, bias)
    dy = rand(T, H, seed=9)
    y.backward(dy)
    return p, y, idx, dy


def test_layer_and_gradients(mods):
    p, y, idx, dy = run(mods)
    q = {k: v.detach().to(f64).requires_grad_(True) for k, v in p.items()}
    want = layer64(q, idx)
    want.backward(dy.to(f64))
    assert float((y.detach().to(f64) - want.detach()).norm() / want.detach().norm()) < 16 * 2.0 ** -8
    for name, v in p.items():
        got, ref = v.grad.to(f64), q[name].grad
        assert v.grad.dtype is v.dtype
        assert float((got - ref).norm() / ref.norm()) < 16 * 2.0 ** -8, name


def test_equal_steps_give_equal_bits(mods):
    p, y, idx, _ = run(mods)
    q, y2, idx2, _ = run(mods)
    assert torch.equal(y, y2) and torch.equal(idx, idx2)
    assert all(torch.equal(p[k].grad, q[k].grad) for k in p)


@pytest.mark.parametrize("name", ["x", "w", "bias", "residual"])
def test_one_gradient_at_a_time(mods, name):
    _, moe = mods
    args = {"x": rand(30, 64, seed=1), "w": rand(44, 64, seed=2, scale=0.1),
            "bias": rand(44, seed=3, dtype=torch.float32), "residual": rand(30, 22, seed=4)}
    dy = rand(30, 22, seed=5)

    def grads(names):
        p = {k: v.clone().requires_grad_(k in names) for k, v in args.items()}
        moe.linear(p["x"], p["w"], p["bias"], "swiglu", p["residual"]).backward(dy)
        return p

    every, one = grads(args), grads([name])
    assert torch.equal(every[name].grad, one[name].grad)
    assert all(one[k].grad is None for k in args if k != name)


def test_strided_arguments(mods):
    ep, moe = mods
    x, w = rand(64, 50, seed=1).t(), rand(64, 24, seed=2).t()
    r = rand(24, 50, seed=3).t()
    assert torch.equal(moe.linear(x, w, residual=r),
                       ep.linear(x.contiguous(), w.contiguous(), residual=r.contiguous()))
    l = rand(32, 20, seed=4).t()
    assert torch.equal(moe.route(l, 3)[0], ep.route(l.contiguous(), 3)[0])
    x2 = x.contiguous().requires_grad_(True)
    moe.linear(x2, w).sum().backward()  # dy is an expanded tensor
    assert torch.allclose(x2.grad.float(), w.float().sum(dim=0).expand(50, 64), rtol=2e-2, atol=2e-2)


@pytest.mark.parametrize("out", [bf, torch.float32])
@pytest.mark.parametrize("act", ["none", "silu"])
def test_arguments_off_16_bytes(mods, out, act):
    """Flat parameters and activations hand out matrices that start anywhere, and so
    does the gradient of a result that was one of several joined ones."""
    _, moe = mods
    x, w, r = rand(5, 64, seed=1), rand(24, 64, seed=2), rand(5, 24, seed=3, dtype=out)
    ones = [t.clone().requires_grad_() for t in (x, w, r)]
    y = moe.linear(ones[0], ones[1], None, act, ones[2], out)
    g = rand(3 + y.numel(), seed=4, dtype=out)
    y.backward(g[3:].view_as(y).clone())
    parts = [torch.cat([t.new_zeros(3), t.flatten()]).requires_grad_() for t in (x, w, r)]
    args = [f[3:].view_as(t) for f, t in zip(parts, (x, w, r))]
    assert all(a.data_ptr() % 16 for a in args)
    got = moe.linear(args[0], args[1], None, act, args[2], out)
    assert torch.equal(got, y)
    torch.cat([got.new_zeros(3), got.flatten()]).backward(g)
    for f, t in zip(parts, ones):
        assert torch.equal(f.grad[3:].view_as(t), t.grad)


def test_without_a_gradient_nothing_is_kept(mods):
    """Parameters ask for a gradient, but not where none is recorded."""
    _, moe = mods
    x, w = rand(512, 256, seed=1), rand(4096, 256, seed=2).requires_grad_()
    with torch.no_grad():
        moe.linear(x, w, activation="silu")  # (the libraries' own first allocations)
        torch.cuda.synchronize()
        torch.cuda.reset_peak_memory_stats()
        before = torch.cuda.memory_allocated()
        y = moe.linear(x, w, activation="silu")
    assert torch.cuda.max_memory_allocated() - before == y.numel() * 2
    assert torch.equal(y, moe.linear(x, w, activation="silu").detach())


def test_second_derivatives_are_refused(mods):
    _, moe = mods
    x = rand(8, 64, seed=1).requires_grad_(True)
    w = rand(16, 64, seed=2)
    g, = torch.autograd.grad(moe.linear(x, w, activation="silu").float().pow(2).sum(), x, create_graph=True)
    with pytest.raises(RuntimeError):
        g.float().sum().backward()
    l = rand(8, 16, seed=3, dtype=torch.float32).requires_grad_(True)
    g, = torch.autograd.grad(moe.route(l, 2)[1].pow(2).sum(), l, create_graph=True)
    with pytest.raises(RuntimeError):
        g.sum().backward()


def test_a_captured_step(mods):
    """Forward and backward in a graph, replayed on other inputs."""
    _, moe = mods
    x, w = rand(40, 64, seed=1).requires_grad_(True), rand(32, 64, seed=2, scale=0.1).requires_grad_(True)
    bias = rand(32, seed=3, dtype=torch.float32).requires_grad_(True)

    def step():
        y = moe.linear(x, w, bias, "silu", out_dtype=torch.float32)
        idx, weights = moe.route(y, 3, None, "sigmoid")
        return idx, torch.autograd.grad(weights.pow(2).sum(), (x, w, bias))

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        idx, grads = step()
    with torch.no_grad():
        x.copy_(rand(40, 64, seed=7))
    graph.replay()
    torch.cuda.synchronize()
    want_idx, want = step()
    assert torch.equal(idx, want_idx)
    assert all(torch.equal(a, b) for a, b in zip(grads, want))
