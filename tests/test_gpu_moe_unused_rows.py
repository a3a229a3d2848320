"""The differentiable movement with receive buffers that hold rows no entry
maps to (masked entries, a buffer of T * K rows): such rows are zero, whatever
the memory held before, so that the experts' gradients see none of it."""
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


def inputs(T, H, E, K, seed, mask):
    inp = W.make_inputs(W.Workload("rows", T=T, H=H, E=E, K=K, seed=seed, mask_frac=mask))
    return inp.x.cuda(), inp.topk_idx.cuda(), inp.topk_w.cuda()


def fill_free_memory(rows, H):
    """Leave NaN in the memory that the next buffers of this size come from."""
    bufs = [torch.full((rows, H), float("nan"), dtype=torch.bfloat16, device="cuda") for _ in range(8)]
    torch.cuda.synchronize()
    del bufs
    probe = torch.empty((rows, H), dtype=torch.bfloat16, device="cuda")
    assert bool(probe.isnan().all()), "the allocator hands out other memory"


@pytest.mark.parametrize("mask", [0.0, 0.2, 1.0])
def test_weight_gradients_with_masked_entries(mods, mask):
    """The experts' weight gradient of the whole composition against 64 bits.
    bf16 rounds each of the four movements and the expert's product (relative
    2^-8 each, rms half of that): 0.02 of the norm."""
    ep, moe = mods
    T, H, E, K = 120, 256, 6, 3
    x, idx, w = inputs(T, H, E, K, seed=3, mask=mask)
    if mask == 1.0:
        idx.fill_(-1)
    _, _, slot = ep.get_dispatch_layout(idx, E)
    g = torch.Generator(device="cuda").manual_seed(1)
    m = (torch.randn((H, H), generator=g, device="cuda") * H ** -0.5).to(torch.bfloat16)
    dy = torch.randn((T, H), generator=g, device="cuda").to(torch.bfloat16)
    for v in (x, w, m):
        v.requires_grad_()
    fill_free_memory(T * K, H)
    moe.combine(moe.dispatch(x, slot, T * K) @ m, slot, w).backward(dy)
    x64, w64, m64 = (v.detach().to(f64).requires_grad_() for v in (x, w, m))
    on = (idx >= 0).to(f64)[..., None]
    (w64[..., None] * on * (x64 @ m64)[:, None]).sum(1).backward(dy.to(f64))
    for got, want in ((x.grad, x64.grad), (w.grad, w64.grad), (m.grad, m64.grad)):
        assert bool(got.isfinite().all())
        assert float((got.to(f64) - want).norm()) <= 0.02 * float(want.norm())


@pytest.mark.parametrize("H", [8, 1000, 4096])
def test_rows_no_entry_maps_to_are_zero(mods, H):
    """Gaps among the used rows and rows past them; the used ones as dispatch
    leaves them."""
    ep, moe = mods
    T, K, spare = 50, 4, 37
    g = torch.Generator(device="cuda").manual_seed(H)
    on = torch.rand((T, K), generator=g, device="cuda") > 0.3
    n = int(on.sum())
    slot = torch.full((T, K), -1, dtype=torch.int32, device="cuda")
    slot[on] = torch.randperm(n + spare, generator=g, device="cuda")[:n].to(torch.int32)
    x = torch.randn((T, H), generator=g, device="cuda").to(torch.bfloat16)
    want = ep.dispatch(x, slot, n + spare)
    used = torch.zeros(n + spare, dtype=torch.bool, device="cuda")
    used[slot[on].long()] = True
    fill_free_memory(n + spare, H)
    got = moe.dispatch(x.requires_grad_(), slot, n + spare)
    assert torch.equal(got[used], want[used]) and bool((got[~used] == 0).all())


def test_no_tokens_and_no_rows(mods):
    _, moe = mods
    x = torch.randn((3, 64), device="cuda").to(torch.bfloat16).requires_grad_()
    slot = torch.full((3, 2), -1, dtype=torch.int32, device="cuda")
    fill_free_memory(6, 64)
    assert bool((moe.dispatch(x[:0], slot[:0], 6) == 0).all())
    out = moe.dispatch(x, slot, 0)
    assert out.shape == (0, 64)
    out.sum().backward()
    assert bool((x.grad == 0).all())
