"""combine's gradient where the weights need none: the expert rows are neither
kept for the backward pass nor needed by the call."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def mods():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    torch.cuda.set_device(0)
    from combine_movement_gb300 import build
    build.build()
    from combine_movement_gb300 import ep, moe
    return ep, moe


def case(T, H, K, seed, spare=4):
    g = torch.Generator(device="cuda").manual_seed(seed)
    on = torch.rand((T, K), generator=g, device="cuda") > 0.1
    n = int(on.sum())
    slot = torch.full((T, K), -1, dtype=torch.int32, device="cuda")
    slot[on] = torch.randperm(n + spare, generator=g, device="cuda")[:n].to(torch.int32)
    rows = torch.randn((n + spare, H), generator=g, device="cuda").to(torch.bfloat16)
    dy = torch.randn((T, H), generator=g, device="cuda").to(torch.bfloat16)
    return rows, slot, torch.rand((T, K), generator=g, device="cuda"), dy


def test_the_rows_are_not_kept(mods):
    _, moe = mods
    rows, slot, w, dy = case(1000, 2048, 4, 1)
    leaf = rows.requires_grad_()
    moe.combine(leaf * 2, slot, w).backward(dy)  # (the allocator's and the library's first uses)
    leaf.grad = None
    torch.cuda.synchronize()
    before = torch.cuda.memory_allocated()
    made = leaf * 2  # (its own backward keeps nothing)
    y = moe.combine(made, slot, w)
    del made
    kept = torch.cuda.memory_allocated() - before
    assert kept < y.numel() * 2 + rows.numel() * 2 // 2, kept
    y.backward(dy)
    frozen = leaf.grad.clone()
    leaf.grad = None
    moe.combine(leaf * 2, slot, w.requires_grad_()).backward(dy)
    assert torch.equal(leaf.grad, frozen)


@pytest.mark.parametrize("T,H,K", [(1, 8, 1), (40, 1000, 3), (500, 4096, 8)])
def test_the_call_without_rows(mods, T, H, K):
    ep, _ = mods
    rows, slot, w, dy = case(T, H, K, T)
    want, got = torch.full_like(rows, 9.0), torch.full_like(rows, 9.0)
    ep.ep_combine_grad(dy, rows, slot, w, want, None)
    ep.ep_combine_grad(dy, None, slot, w, got, None)
    torch.cuda.synchronize()
    assert torch.equal(got, want)


def test_no_rows_at_all(mods):
    """A buffer of no rows has no address: still an output, with nothing in it."""
    ep, moe = mods
    slot = torch.full((5, 2), -1, dtype=torch.int32, device="cuda")
    w = torch.rand((5, 2), device="cuda")
    rows = torch.zeros((0, 64), dtype=torch.bfloat16, device="cuda", requires_grad=True)
    y = moe.combine(rows, slot, w)
    y.sum().backward()
    assert rows.grad.shape == (0, 64) and bool((y == 0).all())
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    slot[3, 1] = 0  # past the end of no rows
    ep.ep_combine_grad(torch.zeros_like(y.detach()), None, slot, w, rows.detach(), None, status)
    assert ep.ep_get_status(status) == ep.EP_ERR_BAD_SLOT
