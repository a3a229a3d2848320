"""Second derivatives through the differentiable dispatch and combine.

Against the same function in 64 bits with torch's own second derivatives. The
sizes are small and every movement rounds to bf16 (relative 2^-8, rms half of
that); a second derivative passes at most six of them (two forward, two
backward, two in the backward's backward), each adding in the mean square:
sqrt(6) * 2^-9 = 0.005 of the norm where terms do not cancel; 0.03 with room
for terms of both signs."""
import pytest
import torch

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


def case(T, H, K, seed, spare=5):
    g = torch.Generator(device="cuda").manual_seed(seed)
    on = torch.rand((T, K), generator=g, device="cuda") > 0.2
    n = int(on.sum())
    slot = torch.full((T, K), -1, dtype=torch.int32, device="cuda")
    slot[on] = torch.randperm(n + spare, generator=g, device="cuda")[:n].to(torch.int32)
    bf = torch.bfloat16
    x = torch.randn((T, H), generator=g, device="cuda").to(bf)
    rows = torch.randn((n + spare, H), generator=g, device="cuda").to(bf)
    w = torch.rand((T, K), generator=g, device="cuda")
    return x, rows, slot, w


def plain_dispatch(x, slot, num_recv):
    at = torch.where(slot < 0, num_recv, slot).long().reshape(-1)
    out = torch.zeros((num_recv + 1, x.shape[1]), dtype=x.dtype, device=x.device)
    return out.index_copy(0, at, x.repeat_interleave(slot.shape[1], 0))[:num_recv]


def plain_combine(rows, slot, w):
    rows = torch.cat([rows, rows.new_zeros((1, rows.shape[1]))])
    at = torch.where(slot < 0, rows.shape[0] - 1, slot).long()
    return (w[..., None] * rows[at]).sum(1)


def close(got, want):
    assert bool(got.isfinite().all())
    assert float((got.to(f64) - want).norm()) <= 0.03 * float(want.norm())


def doubles(*tensors):
    return [t.detach().to(f64).requires_grad_() for t in tensors]


def test_combine(mods):
    """A penalty on both gradients of combine, by the rows, the weights and
    what scales the loss."""
    _, moe = mods
    x, rows, slot, w = case(40, 64, 3, 1)

    def grads(combine, rows, w, s):
        y = combine(rows, slot, w)
        d_rows, d_w = torch.autograd.grad((y * s).pow(2).sum(dtype=f64), (rows, w), create_graph=True)
        loss = d_rows.to(f64).pow(2).sum() + d_w.to(f64).pow(3).sum() + w.to(f64).pow(2).sum()
        return torch.autograd.grad(loss, (rows, w, s))

    s = (x.abs() * 0.3 + 0.3).detach()
    got = grads(moe.combine, rows.requires_grad_(), w.requires_grad_(), s.requires_grad_())
    want = grads(plain_combine, *doubles(rows, w, s))
    for a, b in zip(got, want):
        close(a, b)


def test_combine_of_a_loss_that_is_linear_in_its_result(mods):
    """Its gradient needs none itself, yet d_rows depends on the weights and
    d_w on the rows."""
    _, moe = mods
    _, rows, slot, w = case(40, 64, 3, 2)

    def grads(combine, rows, w):
        y = combine(rows, slot, w)
        d_rows, d_w = torch.autograd.grad(y.sum(dtype=f64), (rows, w), create_graph=True)
        loss = d_rows.to(f64).pow(2).sum() + d_w.to(f64).pow(2).sum()
        return torch.autograd.grad(loss, (rows, w))

    got = grads(moe.combine, rows.requires_grad_(), w.requires_grad_())
    want = grads(plain_combine, *doubles(rows, w))
    for a, b in zip(got, want):
        close(a, b)


@pytest.mark.parametrize("frozen", ["rows", "w"])
def test_combine_with_one_gradient(mods, frozen):
    _, moe = mods
    _, rows, slot, w = case(30, 40, 2, 3)
    wrt = "w" if frozen == "rows" else "rows"

    def grad(combine, rows, w):
        v = {"rows": rows, "w": w}
        v[frozen] = v[frozen].detach()
        y = combine(v["rows"], slot, v["w"])
        (d,) = torch.autograd.grad(y.pow(2).sum(dtype=f64), v[wrt], create_graph=True)
        return torch.autograd.grad(d.to(f64).pow(2).sum() + v[wrt].to(f64).sum(), v[wrt])[0]

    got = grad(moe.combine, rows.requires_grad_(), w.requires_grad_())
    close(got, grad(plain_combine, *doubles(rows, w)))


def test_dispatch(mods):
    _, moe = mods
    x, _, slot, _ = case(40, 64, 3, 4)
    R = int((slot >= 0).sum()) + 5

    def grad(dispatch, x):
        r = dispatch(x, slot, R)
        (dx,) = torch.autograd.grad(r.pow(2).sum(dtype=f64), x, create_graph=True)
        return torch.autograd.grad(dx.to(f64).pow(2).sum() + x.to(f64).pow(2).sum(), x)[0]

    close(grad(moe.dispatch, x.requires_grad_()), grad(plain_dispatch, *doubles(x)))


def test_the_layer_in_training(mods):
    """A penalty on the input's gradient through dispatch, an expert and
    combine, by every parameter."""
    _, moe = mods
    x, _, slot, w = case(50, 64, 3, 5)
    R = slot.numel()
    g = torch.Generator(device="cuda").manual_seed(6)
    m = (torch.randn((64, 64), generator=g, device="cuda") / 8).to(torch.bfloat16)

    def grads(dispatch, combine, x, w, m):
        y = combine(torch.tanh(dispatch(x, slot, R) @ m), slot, w)
        (dx,) = torch.autograd.grad(y.pow(2).sum(dtype=f64), x, create_graph=True)
        return torch.autograd.grad(dx.to(f64).pow(2).sum() + y.sum(dtype=f64), (x, w, m))

    got = grads(moe.dispatch, moe.combine, *(v.requires_grad_() for v in (x, w, m)))
    want = grads(plain_dispatch, plain_combine, *doubles(x, w, m))
    for a, b in zip(got, want):
        close(a, b)


def test_first_derivatives_keep_their_bits_when_a_graph_is_made(mods):
    ep, moe = mods
    x, rows, slot, w = case(40, 64, 3, 7)
    dy = torch.randn_like(x)
    d_rows, d_w = torch.zeros_like(rows), torch.empty_like(w)
    ep.ep_combine_grad(dy, rows, slot, w, d_rows, d_w)
    for create in (False, True):
        y = moe.combine(rows.requires_grad_(), slot, w.requires_grad_())
        got = torch.autograd.grad(y, (rows, w), dy, create_graph=create)
        assert torch.equal(got[0], d_rows) and torch.equal(got[1], d_w)
        r = moe.dispatch(x.requires_grad_(), slot, rows.shape[0])
        (dx,) = torch.autograd.grad(r, x, rows.detach(), create_graph=create)
        assert torch.equal(dx, ep.dispatch_grad(rows.detach(), slot))


def test_inputs_with_strides(mods):
    """Rows and gradients that are not contiguous."""
    _, moe = mods
    x, rows, slot, w = case(30, 64, 2, 8)

    def grads(dispatch, combine, x, rows, w):
        y = combine(rows.T.contiguous().T, slot, w)
        r = dispatch(x.T.contiguous().T, slot, rows.shape[0])
        d = torch.autograd.grad(y.sum(dtype=f64) + (y.T @ y).sum(dtype=f64) + r.pow(2).sum(dtype=f64),
                                (rows, w, x), create_graph=True)
        loss = sum(v.T.to(f64).pow(2).sum() for v in d)
        return (*d, *torch.autograd.grad(loss, (rows, w, x)))

    got = grads(moe.dispatch, moe.combine, *(v.requires_grad_() for v in (x, rows, w)))
    want = grads(plain_dispatch, plain_combine, *doubles(x, rows, w))
    for a, b in zip(got, want):
        close(a.detach(), b.detach())
