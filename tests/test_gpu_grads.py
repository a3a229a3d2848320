"""The gradients of dispatch and combine against the formulas in 64 bits and
against differences of the 64-bit forward.

Tolerances. d_expert_out is one fp32 product rounded to bf16: (1 + 2^-24) and
half a unit of 8 significant bits, together below 2^-8 + 2^-23 of the value.
d_topk_w sums H products in fp32 in some order, each addition (and product)
off by at most 2^-24 of the magnitudes so far: H * 2^-24 * sum|p| covers it.
dx sums K values: K * 2^-24 * sum|v|, and the rounding to bf16.
"""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu
f64 = torch.float64


@pytest.fixture(scope="module")
def ep():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    torch.cuda.set_device(0)
    from combine_movement_gb300 import build
    build.build()
    from combine_movement_gb300 import ep as mod
    yield mod
    mod.ep_set_num_sms(0)


def case(T, H, K, seed, mask=0.0, spare=0):
    """dy, expert rows, slot, weights: slots are a random placement of the
    unmasked entries, with `spare` unused rows among them."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    on = torch.rand((T, K), generator=g, device="cuda") >= mask
    n = int(on.sum())
    rows = torch.randperm(n + spare, generator=g, device="cuda")[:n].to(torch.int32)
    slot = torch.full((T, K), -1, dtype=torch.int32, device="cuda")
    slot[on] = rows
    dy = torch.randn((T, H), generator=g, device="cuda").to(torch.bfloat16)
    e = torch.randn((n + spare, H), generator=g, device="cuda").to(torch.bfloat16)
    w = torch.randn((T, K), generator=g, device="cuda")
    return dy, e, slot, w


def gathered(rows, slot):
    """fp64 [T, K, H] of the slots' rows, zeros where masked."""
    pad = torch.cat([rows.to(f64), rows.new_zeros((1, rows.shape[1])).to(f64)])
    return pad[torch.where(slot < 0, rows.shape[0], slot).long()]


def check(ep, T, H, K, seed, mask=0.0, spare=0, num_sms=0):
    dy, e, slot, w = case(T, H, K, seed, mask, spare)
    de = torch.full_like(e, 9.0)
    dw = torch.full_like(w, 9.0)
    dx = torch.full_like(dy, 9.0)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    ep.ep_set_num_sms(num_sms)
    ep.ep_combine_grad(dy, e, slot, w, de, dw, status)
    ep.ep_dispatch_grad(e, slot, dx, status)
    ep.ep_set_num_sms(0)
    assert ep.ep_get_status(status) == ep.EP_OK
    rows = gathered(e, slot)
    p = dy.to(f64)[:, None] * rows
    assert bool(((dw.to(f64) - p.sum(2)).abs() <= H * 2.0 ** -24 * p.abs().sum(2)).all())
    want = w.to(f64)[..., None] * dy.to(f64)[:, None]
    on = slot >= 0
    got = de[slot[on].long()].to(f64)
    assert bool(((got - want[on]).abs() <= want[on].abs() * (2.0 ** -8 + 2.0 ** -23)).all())
    untouched = torch.ones(e.shape[0], dtype=torch.bool, device="cuda")
    untouched[slot[on].long()] = False
    assert bool((de[untouched] == 9.0).all())
    s = rows.sum(1)
    tol = s.abs() * (2.0 ** -8 + 2.0 ** -23) + K * 2.0 ** -23 * rows.abs().sum(1)
    assert bool(((dx.to(f64) - s).abs() <= tol).all())


@pytest.mark.parametrize("H", [8, 64, 248, 256, 264, 1000, 1032, 2048, 7168])
@pytest.mark.parametrize("K", [1, 2, 8])
def test_widths(ep, H, K):
    check(ep, 37, H, K, seed=H + K, mask=0.2, spare=3)


@pytest.mark.parametrize("T,K,H", [(1, 1, 8), (1, 8, 7168), (2, 32, 4096), (3, 9, 16384),
                                   (300, 6, 4096), (1500, 3, 2056), (5, 31, 40)])
def test_shapes(ep, T, K, H):
    check(ep, T, H, K, seed=T + K, mask=0.1)


@pytest.mark.parametrize("num_sms", [1, 24])
def test_sm_budget(ep, num_sms):
    check(ep, 200, 1024, 4, seed=5, mask=0.1, spare=7, num_sms=num_sms)


def test_large(ep):
    check(ep, 2048, 7168, 8, seed=6)


def test_everything_masked(ep):
    dy, e, slot, w = case(20, 512, 4, seed=1, mask=2.0, spare=8)
    assert bool((slot == -1).all())
    de, dw = torch.full_like(e, 9.0), torch.full_like(w, 9.0)
    ep.ep_combine_grad(dy, e, slot, w, de, dw)
    assert bool((dw == 0).all()) and bool((de == 9.0).all())
    assert bool((ep.dispatch_grad(e, slot) == 0).all())


def test_no_tokens(ep):
    dy, e, slot, w = case(4, 64, 2, seed=1)
    de, dw = ep.combine_grad(dy[:0], e, slot[:0], w[:0])
    assert de.shape == e.shape and dw.shape == (0, 2)
    assert ep.dispatch_grad(e, slot[:0]).shape == (0, 64)


def test_one_output_at_a_time(ep):
    dy, e, slot, w = case(50, 1000, 5, seed=2, mask=0.3)
    de, dw = ep.combine_grad(dy, e, slot, w)
    only_e, only_w = torch.empty_like(de), torch.empty_like(dw)
    ep.ep_combine_grad(dy, e, slot, w, only_e, None)
    ep.ep_combine_grad(dy, e, slot, w, None, only_w)
    on = slot[slot >= 0].long()
    assert torch.equal(only_e[on], de[on]) and torch.equal(only_w, dw)


def test_slots_past_the_buffer_are_reported_and_skipped(ep):
    dy, e, slot, w = case(30, 256, 3, seed=3)
    slot[4, 1] = e.shape[0]
    de, dw = torch.full_like(e, 9.0), torch.full_like(w, 9.0)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    ep.ep_combine_grad(dy, e, slot, w, de, dw, status)
    assert ep.ep_get_status(status) == ep.EP_ERR_BAD_SLOT
    assert float(dw[4, 1]) == 0 and bool((dw[5:] != 9.0).all())
    status.zero_()
    dx = torch.empty_like(dy)
    ep.ep_dispatch_grad(e, slot, dx, status)
    assert ep.ep_get_status(status) == ep.EP_ERR_BAD_SLOT


def test_values_that_are_not_finite_stay_in_their_entries(ep):
    dy, e, slot, w = case(10, 512, 2, seed=4)
    e[slot[3, 1].long(), 7] = float("nan")
    dy[6, 0] = float("inf")
    de, dw = ep.combine_grad(dy, e, slot, w)
    bad = torch.zeros_like(dw, dtype=torch.bool)
    bad[3, 1] = True
    bad[6] = True
    assert bool((dw.isfinite() == ~bad).all())
    rows = de.isfinite().all(1)[slot.long()]
    assert bool((rows == ~(torch.arange(10, device="cuda") == 6)[:, None]).all())


def test_same_bits_every_time_and_on_another_stream(ep):
    dy, e, slot, w = case(400, 4096, 6, seed=7)
    first = ep.combine_grad(dy, e, slot, w)
    dx = ep.dispatch_grad(e, slot)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        again = ep.combine_grad(dy, e, slot, w)
        dx2 = ep.dispatch_grad(e, slot)
    torch.cuda.synchronize()
    assert torch.equal(again[0], first[0]) and torch.equal(again[1], first[1])
    assert torch.equal(dx2, dx)


def test_against_differences(ep):
    """The forward is linear in the rows and in the weights, so a central
    difference of any step is its derivative but for rounding in 64 bits."""
    T, H, K = 6, 48, 3
    dy, e, slot, w = case(T, H, K, seed=8, mask=0.2, spare=2)
    de, dw = ep.combine_grad(dy, e, slot, w)
    dx = ep.dispatch_grad(e, slot)
    e_, w_, dy_ = e.to(f64), w.to(f64), dy.to(f64)

    def loss(rows, weights):
        return float((dy_ * (weights[..., None] * gathered(rows, slot)).sum(1)).sum())

    rng = np.random.default_rng(0)
    step = 0.5
    for t in range(T):
        for k in range(K):
            d = torch.zeros_like(w_)
            d[t, k] = step
            diff = (loss(e_, w_ + d) - loss(e_, w_ - d)) / (2 * step)
            assert abs(diff - float(dw[t, k])) <= 1e-4 * max(1.0, abs(diff))
    used = slot[slot >= 0].tolist()
    for r in rng.choice(used, 6, replace=False):
        h = int(rng.integers(H))
        d = torch.zeros_like(e_)
        d[int(r), h] = step
        diff = (loss(e_ + d, w_) - loss(e_ - d, w_)) / (2 * step)
        assert abs(diff - float(de[int(r), h])) <= 2.0 ** -8 * abs(diff) + 1e-9
    x = torch.randn((T, H), dtype=f64, device="cuda")

    def moved(x):  # <e, dispatch(x)> with e as the gradient of the receive rows
        return float((x[:, None] * gathered(e, slot)).sum())

    for _ in range(6):
        t, h = int(rng.integers(T)), int(rng.integers(H))
        d = torch.zeros_like(x)
        d[t, h] = step
        diff = (moved(x + d) - moved(x - d)) / (2 * step)
        assert abs(diff - float(dx[t, h])) <= 2.0 ** -8 * abs(diff) + 1e-9
