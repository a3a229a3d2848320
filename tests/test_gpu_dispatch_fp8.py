"""The quantising dispatch against the definition in 64 bits. The scale is one
correctly rounded fp32 division, so it is compared bit for bit (a division in
64 bits rounded to fp32 is the fp32 division). A value times the rounded
inverse, rounded, is off by 2^-23 before it goes to e4m3, which rounds to
4 significant bits (2^-4) or half its smallest step (2^-10 of the scale)."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu
f64 = torch.float64
F8 = torch.float8_e4m3fn


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


def routed(T, K, seed, mask=0.0, spare=0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    on = torch.rand((T, K), generator=g, device="cuda") >= mask
    n = int(on.sum())
    slot = torch.full((T, K), -1, dtype=torch.int32, device="cuda")
    slot[on] = torch.randperm(n + spare, generator=g, device="cuda")[:n].to(torch.int32)
    return slot, n + spare


def blocks64(x):
    """fp64 [T, blocks, 128] with zeros past the width."""
    return torch.nn.functional.pad(x.to(f64), (0, -x.shape[1] % 128)).unflatten(1, (-1, 128))


def check(ep, x, slot, R, num_sms=0):
    T, H = x.shape
    K = slot.shape[1]
    w = torch.rand((T, K), device="cuda")
    q = torch.full((R, H), 5.0, device="cuda").to(F8)
    s = torch.full((R, -(-H // 128)), 5.0, device="cuda")
    rw = torch.full((R,), 5.0, device="cuda")
    rs = torch.full((R,), -5, dtype=torch.int32, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    ep.ep_set_num_sms(num_sms)
    ep.ep_dispatch_fp8(x, slot, q, s, w, rw, rs, status)
    ep.ep_set_num_sms(0)
    assert ep.ep_get_status(status) == ep.EP_OK
    b = blocks64(x)
    m = b.abs().amax(2).clamp_min(float(np.float32(1e-30)))
    want_s = (m / 448).to(torch.float32)
    t, k = (slot >= 0).nonzero(as_tuple=True)
    r = slot[t, k].long()
    assert torch.equal(s[r], want_s[t])
    step = want_s.to(f64)[t][..., None]
    err = (blocks64(q[r].to(f64)) * step - b[t]).abs()
    assert bool((err <= b[t].abs() * (2.0 ** -4 + 2.0 ** -20) + step * 2.0 ** -10).all())
    top = blocks64(q[r].to(f64)).abs().amax(2)
    assert bool((top[m[t] > 1e-29] == 448).all())
    assert torch.equal(rw[r], w[t, k]) and torch.equal(rs[r], (t * K + k).to(torch.int32))
    rest = torch.ones(R, dtype=torch.bool, device="cuda")
    rest[r] = False
    assert bool((q[rest].float() == 5).all()) and bool((s[rest] == 5).all())
    assert bool((rw[rest] == 5).all()) and bool((rs[rest] == -5).all())


def rows(T, H, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    x = torch.randn((T, H), generator=g, device="cuda")
    return (x * torch.exp(2 * torch.randn((T, 1), generator=g, device="cuda"))).to(torch.bfloat16)


@pytest.mark.parametrize("H", [16, 112, 128, 144, 496, 512, 528, 1024, 1040, 7168])
@pytest.mark.parametrize("K", [1, 8])
def test_widths(ep, H, K):
    slot, R = routed(41, K, H + K, mask=0.2, spare=4)
    check(ep, rows(41, H, H), slot, R)


@pytest.mark.parametrize("T,K,H,num_sms", [(1, 8, 7168, 0), (1, 1, 16, 0), (7, 32, 256, 0),
                                           (3000, 4, 2048, 0), (6000, 8, 4096, 0),
                                           (500, 6, 1040, 1), (2000, 8, 7168, 24)])
def test_shapes(ep, T, K, H, num_sms):
    slot, R = routed(T, K, T, mask=0.05)
    check(ep, rows(T, H, T), slot, R, num_sms)


def test_extreme_values(ep):
    x = torch.zeros((6, 256), device="cuda", dtype=torch.bfloat16)
    x[1] = 3.0e38
    x[2, 3] = 1e-38                       # below the floor: zeros, the floor's scale
    x[3] = torch.linspace(-1, 1, 256)
    x[4, 200] = -2.0 ** -100
    x[5] = 1e-29
    slot, R = routed(6, 2, 3)
    check(ep, x, slot, R)


def test_values_that_are_not_finite_show_in_their_block(ep):
    x = rows(3, 384, 1)
    x[1, 130] = float("inf")
    x[2, 5] = float("nan")
    slot = torch.arange(3, dtype=torch.int32, device="cuda")[:, None]
    q, s = ep.dispatch_fp8(x, slot, 3)
    bad = torch.zeros((3, 3), dtype=torch.bool, device="cuda")
    bad[1, 1] = bad[2, 0] = True
    assert bool((s.isfinite() == ~bad).all())
    value = q.float().unflatten(1, (3, 128)) * s[..., None]
    assert bool((value.isfinite().all(2) == ~bad).all())
    assert not bool(value[bad].isfinite().any())


def test_no_tokens_and_everything_masked(ep):
    x = rows(4, 128, 1)
    slot = torch.full((4, 2), -1, dtype=torch.int32, device="cuda")
    q = torch.full((3, 128), 5.0, device="cuda").to(F8)
    s = torch.full((3, 1), 5.0, device="cuda")
    ep.ep_dispatch_fp8(x, slot, q, s)
    ep.ep_dispatch_fp8(x[:0], slot[:0], q, s)
    assert bool((q.float() == 5).all()) and bool((s == 5).all())


def test_slots_past_the_buffer_are_reported_and_skipped(ep):
    x = rows(40, 256, 2)
    slot, R = routed(40, 3, 5)
    q0, s0 = ep.dispatch_fp8(x, slot, R)
    short = slot.clone()
    q = torch.zeros((R - 2, 256), device="cuda").to(F8)
    s = torch.zeros((R - 2, 2), device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    ep.ep_dispatch_fp8(x, short, q, s, status=status)
    assert ep.ep_get_status(status) == ep.EP_ERR_BAD_SLOT
    assert torch.equal(q.view(torch.uint8), q0.view(torch.uint8)[:R - 2])
    assert torch.equal(s, s0[:R - 2])


def test_same_bits_every_time_and_on_another_stream(ep):
    x = rows(700, 2048, 3)
    slot, R = routed(700, 4, 6)
    q0, s0 = ep.dispatch_fp8(x, slot, R)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        q1, s1 = ep.dispatch_fp8(x, slot, R)
    torch.cuda.synchronize()
    assert torch.equal(q0.view(torch.uint8), q1.view(torch.uint8)) and torch.equal(s0, s1)
