"""The gated product's activation over the range of its gate, from where
exp(-g) overflows to where it vanishes, infinities included.

One row value of 1 and one weight of 1 in each column make a block's gate and
up the weight blocks' scales exactly, so that h = silu(g) u shows in the
output's scale (h is constant over the block: scale = |h| / 448, q = +-448).

Tolerance, relative to |h|: CUDA's documentation gives __expf(x) 2 +
floor(1.173 |x|) units of 2^-23 and __fdividef 2 units for denominators up to
2^126; the products and sums before and after are four roundings of half a
unit, and a rounded g would move h by |g| / 2 units more; the scale's division
half a unit: below (8 + 2 |g|) 2^-23. Where exp(-|g|) is below 2^-126 it and
its product with g are multiples of 2^-149, off by half of one each:
|u| (|g| + 1) 2^-149, and one more for the product with u's rounding, which
2^-148 (|g| + 1) |u| covers. Values under 1e-30 show as the quantiser's
floor."""
import pytest
import torch

pytestmark = pytest.mark.gpu

F8 = torch.float8_e4m3fn
f64 = torch.float64
FLOOR = float(torch.tensor(1e-30, dtype=torch.float32))


@pytest.fixture(scope="module")
def ep():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    torch.cuda.set_device(0)
    from combine_movement_gb300 import build
    build.build()
    from combine_movement_gb300 import ep as mod
    return mod


def gated(ep, gates, ups, K, rows=3):
    """(q, scale) of blocks with these gates and ups, one for each."""
    n = len(gates)
    a = torch.zeros((rows, K), device="cuda")
    a[:, 0] = 1
    a_scale = torch.ones((rows, -(-K // 128)), device="cuda")
    w = torch.zeros((1, 2 * 128 * n, K), device="cuda")
    w[:, :, 0] = 1
    w_scale = torch.ones((1, 2 * n, -(-K // 128)), device="cuda")
    w_scale[0, :, 0] = torch.tensor(gates + ups, device="cuda")
    offsets = torch.tensor([0, rows], dtype=torch.int32, device="cuda")
    return ep.expert_gate_up_fp8(a.to(F8), a_scale, offsets, w.to(F8), w_scale)


GATES = [-200.0, -103.0, -100.0, -95.5, -89.0, -88.73, -88.5, -88.0, -87.5, -87.34, -87.3, -87.0,
         -80.0, -60.25, -20.0, -5.5, -1.0, -2.0 ** -20, 0.0, 2.0 ** -20, 1.0, 5.5, 20.0, 80.0, 87.5,
         88.5, 89.0, 200.0, 1e30]


# the second splits a tile's K over a cluster of CTAs
@pytest.mark.parametrize("K", [128, 7168])
@pytest.mark.parametrize("u", [1e12, -3.0])
def test_gates(ep, K, u):
    # (the up is as large as keeps h finite)
    ups = [u if abs(g) < 1e20 else u * 1e-10 for g in GATES]
    q, scale = gated(ep, GATES, ups, K)
    g = torch.tensor(GATES, device="cuda").to(f64)
    up = torch.tensor(ups, device="cuda").to(f64)
    h = g / (1 + torch.exp(-g)) * up
    got = scale.to(f64) * 448
    tol = h.abs() * (8 + 2 * g.abs().clamp_max(1e3)) * 2.0 ** -23 + (g.abs().clamp_max(1e3) + 1) * \
        up.abs() * 2.0 ** -148
    want = h.abs().clamp_min(FLOOR)
    assert bool(((got - want).abs() <= tol + want * 2.0 ** -22).all()), (got - want, tol)
    shown = h.abs() > 2 * FLOOR
    shown &= tol < 0.5 * h.abs()
    assert int(shown.sum()) >= 15
    value = q.view(torch.uint8).view(F8).to(f64).unflatten(1, (-1, 128))
    expect = 448 * torch.sign(h)[None, :, None].expand_as(value)
    assert torch.equal(value[:, shown], expect[:, shown])


@pytest.mark.parametrize("K", [128, 7168])
def test_gates_that_are_not_finite(ep, K):
    """silu(inf) = inf; the formula has no value at -inf and NaN. Each shows in
    its block's scale alone."""
    inf, nan = float("inf"), float("nan")
    gates = [inf, 2.0, -inf, -3.0, nan, 0.5]
    q, scale = gated(ep, gates, [2.0] * 6, K)
    assert bool((scale.isfinite() == torch.tensor([False, True] * 3, device="cuda")).all())
    clean_q, clean = gated(ep, [1.0, 2.0, 1.0, -3.0, 1.0, 0.5], [2.0] * 6, K)
    assert torch.equal(scale[:, 1::2], clean[:, 1::2])


@pytest.mark.parametrize("K", [256, 7168])
def test_columns_of_one_block_with_many_gates(ep, K):
    """A block's columns from -96 to 96 at once: its scale is the largest's,
    the rest rounds to e4m3 (2^-4 of the value, or half the smallest step)."""
    cols = torch.arange(128, device="cuda") * 1.5 - 96
    w = torch.zeros((1, 256, K), device="cuda")
    w[0, :128, 0], w[0, :128, 1] = (cols / 8).round(), cols - 8 * (cols / 8).round()
    w[0, 128:, 2] = torch.where(torch.arange(128, device="cuda") % 3 == 0, -1.0, 1.0)
    assert torch.equal(w.to(F8).float(), w)
    a = torch.zeros((5, K), device="cuda")
    a[:, 0], a[:, 1], a[:, 2] = 8, 1, 2
    kb = -(-K // 128)
    offsets = torch.tensor([0, 5], dtype=torch.int32, device="cuda")
    q, scale = ep.expert_gate_up_fp8(a.to(F8), torch.ones((5, kb), device="cuda"), offsets, w.to(F8),
                                     torch.ones((1, 2, kb), device="cuda"))
    g = cols.to(f64)
    h = g / (1 + torch.exp(-g)) * 2 * w[0, 128:, 2].to(f64)
    top = float(h.abs().max())
    assert bool(((scale.to(f64) * 448 - top).abs() <= top * (9 + 2 * 96) * 2.0 ** -23).all())
    step = scale.to(f64)
    err = (q.to(f64) * step - h).abs()
    assert bool((err <= h.abs() * (2.0 ** -4 + (10 + 2 * g.abs()) * 2.0 ** -23) + step * 2.0 ** -10).all())
