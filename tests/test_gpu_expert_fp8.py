"""The experts' 8-bit products against the formula in 64 bits.

Tolerances. A block of 128 products is summed by the tensor core and the
blocks in fp32; each of the at most 128 + ceil(K/128) additions may lose one
unit of 2^-23 of the sum of magnitudes so far, so a sum of products p_i is
within (128 + ceil(K/128)) * 2^-23 * sum|p_i| of its exact value. bf16 output
adds half a unit of its 8 significant bits, 2^-8 |y|. For h = silu(g) * u that error goes through the
derivative (|silu'| < 1.1, |silu(g)| <= |g|), plus 16 units of 2^-24 |h| for
the exponential, the division and the products. An e4m3 value is within
2^-4 of what was rounded, or half the smallest step, 2^-10, of the scale.
"""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

F8 = torch.float8_e4m3fn
f64 = torch.float64


@pytest.fixture(scope="module")
def ep():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    torch.cuda.set_device(0)
    from combine_movement_gb300 import build
    build.build()
    from combine_movement_gb300 import ep as mod
    return mod


def operands(counts, N, K, seed, spare=0):
    """Random rows and weights for these per-expert row counts, with `spare`
    rows past the last expert's."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    E, R = len(counts), sum(counts) + spare
    kb, nb = -(-K // 128), -(-N // 128)

    def fp8(*shape):
        v = torch.randn(shape, generator=g, device="cuda") * 109
        return v.clamp_(-448, 448).to(F8)

    def scales(*shape):
        return torch.randn(shape, generator=g, device="cuda").mul_(0.5).exp_() / 109

    offsets = torch.zeros(E + 1, dtype=torch.int32)
    offsets[1:] = torch.tensor(counts).cumsum(0)
    return (fp8(R, K), scales(R, kb), offsets.cuda(), fp8(E, N, K),
            scales(E, nb, kb) * K ** -0.5)


def spread(scale, K):
    return scale.to(f64).repeat_interleave(128, dim=-1)[..., :K]


def product64(a, a_scale, counts, w, w_scale):
    """(y, bound on its fp32 error) for the rows of every expert, in 64 bits."""
    K, N = a.shape[1], w.shape[1]
    a64 = a.to(f64) * spread(a_scale, K)
    y = torch.zeros((a.shape[0], N), dtype=f64, device=a.device)
    mag = torch.zeros_like(y)
    r = 0
    for e, m in enumerate(counts):
        w64 = w[e].to(f64) * spread(w_scale[e], K).repeat_interleave(128, dim=0)[:N]
        y[r:r + m] = a64[r:r + m] @ w64.T
        mag[r:r + m] = a64[r:r + m].abs() @ w64.abs().T
        r += m
    return y, mag * (128 + -(-K // 128)) * 2.0 ** -23


def check_matmul(ep, counts, N, K, seed=0, spare=0):
    a, a_scale, offsets, w, w_scale = operands(counts, N, K, seed, spare)
    out = torch.full((a.shape[0], N), 777.0, dtype=torch.bfloat16, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    ep.ep_expert_matmul_fp8(a, a_scale, offsets, w, w_scale, out, status)
    assert ep.ep_get_status(status) == ep.EP_OK
    y, tol = product64(a, a_scale, counts, w, w_scale)
    R = sum(counts)
    err = (out[:R].to(f64) - y[:R]).abs()
    assert bool((err <= y[:R].abs() * 2.0 ** -8 + tol[:R] * 1.01).all()), float((err - tol[:R]).max())
    assert bool((out[R:] == 777.0).all()), "rows past the last expert's were written"


@pytest.mark.parametrize("K", [16, 112, 128, 144, 1072, 2048])
def test_inner_sizes(ep, K):
    check_matmul(ep, [5, 0, 130, 1], 264, K, seed=K)


@pytest.mark.parametrize("N", [8, 120, 128, 136, 256, 264, 1000])
def test_output_widths(ep, N):
    check_matmul(ep, [3, 17, 0, 200], N, 272, seed=N, spare=3)


@pytest.mark.parametrize("counts", [
    [1], [0, 0, 1], [127], [128], [129], [255, 256, 257], [16, 17, 32, 33, 64, 65],
    [0] * 40 + [700] + [0] * 23, [1] * 300, [0, 513, 0, 0, 2, 0],
])
def test_row_counts(ep, counts):
    check_matmul(ep, counts, 384, 384, seed=len(counts))


def test_many_experts(ep):
    rng = np.random.default_rng(4)
    check_matmul(ep, list(rng.integers(0, 4, 4096)), 128, 128, seed=9)


def test_deep_and_wide(ep):
    check_matmul(ep, [300, 10, 90, 0], 7168, 2048, seed=5)
    check_matmul(ep, [33, 140], 1024, 7168, seed=6)


def test_no_rows(ep):
    a, a_scale, offsets, w, w_scale = operands([0, 0], 128, 128, 1, spare=4)
    out = torch.full((4, 128), 5.0, dtype=torch.bfloat16, device="cuda")
    ep.ep_expert_matmul_fp8(a, a_scale, offsets, w, w_scale, out)
    assert bool((out == 5.0).all())
    empty = ep.expert_matmul_fp8(a[:0], a_scale[:0], offsets, w, w_scale)
    assert empty.shape == (0, 128)


def check_gate_up(ep, counts, width, K, seed=0, spare=0):
    a, a_scale, offsets, w, w_scale = operands(counts, 2 * width, K, seed, spare)
    R = sum(counts)
    q = torch.full((a.shape[0], width), 3.0, device="cuda").to(F8)
    scale = torch.full((a.shape[0], width // 128), 3.0, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    ep.ep_expert_gate_up_fp8(a, a_scale, offsets, w, w_scale, q, scale, status)
    assert ep.ep_get_status(status) == ep.EP_OK
    y, tol = product64(a, a_scale, counts, w, w_scale)
    g, u, dg, du = y[:R, :width], y[:R, width:], tol[:R, :width], tol[:R, width:]
    h = g * torch.sigmoid(g) * u
    dh = 1.1 * dg * (u.abs() + du) + (g.abs() + dg) * du + h.abs() * 16 * 2.0 ** -24
    amax = h.abs().unflatten(1, (-1, 128)).amax(2)
    damax = dh.unflatten(1, (-1, 128)).amax(2)
    s64 = scale[:R].to(f64)
    assert bool(((s64 - amax / 448).abs() <= damax / 448 + amax / 448 * 2.0 ** -23).all())
    value = q[:R].to(f64) * spread(scale[:R], width)
    step = spread(scale[:R], width)
    assert bool(((value - h).abs() <= h.abs() * 2.0 ** -4 + step * 2.0 ** -10 + 1.1 * dh).all())
    # the block's largest value is at the top of the range
    top = q[:R].to(f64).abs().unflatten(1, (-1, 128)).amax(2)
    assert bool((top == 448).all())
    assert bool((q[R:].float() == 3.0).all()) and bool((scale[R:] == 3.0).all())


@pytest.mark.parametrize("width", [128, 256, 640])
@pytest.mark.parametrize("K", [48, 256, 1040])
def test_gate_up(ep, width, K):
    check_gate_up(ep, [4, 0, 129, 300], width, K, seed=width + K, spare=2)


def test_gate_up_large(ep):
    check_gate_up(ep, [1, 0, 70, 130, 256, 3], 2048, 7168, seed=8)


def test_zero_rows_and_weights(ep):
    a, a_scale, offsets, w, w_scale = operands([6], 256, 256, 2)
    a[2] = 0
    a_scale[3] = 0
    q, scale = ep.expert_gate_up_fp8(a, a_scale, offsets, w, w_scale)
    floor = np.float32(1e-30) / np.float32(448)
    for r in (2, 3):
        assert bool((q[r].float() == 0).all()) and float(scale[r, 0]) == floor
    assert bool((scale[[0, 1, 4, 5]] > 1e-6).all())


def test_values_that_are_not_finite_stay_in_their_row(ep):
    counts = [40, 10]
    a, a_scale, offsets, w, w_scale = operands(counts, 256, 256, 3)
    clean = ep.expert_matmul_fp8(a, a_scale, offsets, w, w_scale)
    qc, sc = ep.expert_gate_up_fp8(a, a_scale, offsets, w, w_scale)
    a.view(torch.uint8)[7, 5] = 0x7F  # e4m3 NaN
    a_scale[45, 1] = float("inf")
    out = ep.expert_matmul_fp8(a, a_scale, offsets, w, w_scale)
    q, s = ep.expert_gate_up_fp8(a, a_scale, offsets, w, w_scale)
    hit = torch.zeros(50, dtype=torch.bool, device="cuda")
    hit[[7, 45]] = True
    assert not bool(out[hit].isfinite().any()) and not bool(s[hit].isfinite().any())
    assert torch.equal(out[~hit], clean[~hit])
    assert torch.equal(q.view(torch.uint8)[~hit], qc.view(torch.uint8)[~hit])
    assert torch.equal(s[~hit], sc[~hit])


def test_repeatable_and_on_another_stream(ep):
    counts = [200, 0, 77, 500]
    a, a_scale, offsets, w, w_scale = operands(counts, 1024, 1024, 12)
    first = ep.expert_matmul_fp8(a, a_scale, offsets, w, w_scale)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        again = [ep.expert_matmul_fp8(a, a_scale, offsets, w, w_scale) for _ in range(5)]
    other = ep.expert_matmul_fp8(a, a_scale, offsets, w, w_scale, stream=side)
    torch.cuda.synchronize()
    for x in again + [other]:
        assert torch.equal(x, first)


def test_bad_offsets_are_reported_and_skipped(ep):
    a, a_scale, offsets, w, w_scale = operands([10, 20, 30], 128, 128, 5)
    good = ep.expert_matmul_fp8(a, a_scale, offsets, w, w_scale)
    bad = offsets.clone()
    bad[3] = 61  # one row more than there are
    out = torch.zeros_like(good)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    ep.ep_expert_matmul_fp8(a, a_scale, bad, w, w_scale, out, status)
    assert ep.ep_get_status(status) == ep.EP_ERR_BAD_SLOT
    assert torch.equal(out[:30], good[:30]) and bool((out[30:] == 0).all())
    bad = offsets.clone()
    bad[1] = -4
    out.zero_()
    status.zero_()
    ep.ep_expert_matmul_fp8(a, a_scale, bad, w, w_scale, out, status)
    assert ep.ep_get_status(status) == ep.EP_ERR_BAD_SLOT
    assert torch.equal(out[30:], good[30:]) and bool((out[:30] == 0).all())


def test_in_a_cuda_graph(ep):
    counts = [64, 3, 0, 150]
    a, a_scale, offsets, w, w_scale = operands(counts, 512, 512, 21)
    want = ep.expert_matmul_fp8(a, a_scale, offsets, w, w_scale)
    out = torch.zeros_like(want)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ep.ep_expert_matmul_fp8(a, a_scale, offsets, w, w_scale, out)
    for _ in range(3):
        out.zero_()
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)


@pytest.mark.parametrize("seed", range(12))
def test_random_shapes(ep, seed):
    """Random per-expert counts (many empty, a few large), widths and depths."""
    rng = np.random.default_rng(seed)
    E = int(rng.integers(1, 80))
    counts = [int(c) for c in rng.integers(0, 300, E) * (rng.random(E) < 0.5)]
    counts[int(rng.integers(E))] += 1
    K = 16 * int(rng.integers(1, 80))
    check_matmul(ep, counts, 8 * int(rng.integers(1, 100)), K, seed=seed, spare=int(rng.integers(5)))
    check_gate_up(ep, counts, 128 * int(rng.integers(1, 5)), K, seed=seed, spare=int(rng.integers(5)))


def test_overlapping_offsets_stay_in_bounds(ep):
    """Offsets that go back are reported; whatever is written stays inside."""
    a, a_scale, offsets, w, w_scale = operands([40, 40, 40, 40], 128, 128, 5, spare=8)
    bad = torch.tensor([0, 160, 0, 160, 160], dtype=torch.int32, device="cuda")
    out = torch.zeros((168, 128), dtype=torch.bfloat16, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    ep.ep_expert_matmul_fp8(a, a_scale, bad, w, w_scale, out, status)
    assert ep.ep_get_status(status) == ep.EP_ERR_BAD_SLOT
    assert bool((out[160:] == 0).all())
