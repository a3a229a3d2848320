"""Few, deep tiles of the experts' products, whose blocks along K a cluster of
CTAs shares: the same formulas and tolerances as for the others (the parts'
sums are joined in fp32, so a sum is still at most 128 + ceil(K/128) additions
deep)."""
import pytest
import torch

from test_gpu_expert_fp8 import check_gate_up, check_matmul, operands

pytestmark = pytest.mark.gpu

F8 = torch.float8_e4m3fn


@pytest.fixture(scope="module")
def ep():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    torch.cuda.set_device(0)
    from combine_movement_gb300 import build
    build.build()
    from combine_movement_gb300 import ep as mod
    return mod


# one tile, a few, as many as share in fours, in twos; the last column tile cut
@pytest.mark.parametrize("counts, N", [
    ([1], 8), ([1], 256), ([1], 1000), ([0, 0, 1, 0], 136), ([1, 1], 2048), ([0, 3], 7168),
    ([1] * 8, 1024), ([2, 0, 1], 5000), ([17, 5], 264), ([128], 256), ([129], 512),
    ([127, 0, 3, 130], 768), ([300], 1024),
])
@pytest.mark.parametrize("K", [1792, 2064, 3056, 7168])
def test_products(ep, counts, N, K):
    check_matmul(ep, counts, N, K, seed=len(counts) + N + K)


@pytest.mark.parametrize("counts, width", [
    ([1], 128), ([1], 2048), ([0, 0, 2], 640), ([1] * 6, 256), ([33], 128), ([128], 256),
    ([129, 0, 7], 384),
])
@pytest.mark.parametrize("K", [1792, 2064, 3200, 7168])
def test_gate_up(ep, counts, width, K):
    check_gate_up(ep, counts, width, K, seed=len(counts) + width + K)


@pytest.mark.parametrize("spare", [1, 40, 500])
def test_rows_past_the_last_are_kept(ep, spare):
    check_matmul(ep, [3, 0, 2], 520, 4096, seed=spare, spare=spare)
    check_gate_up(ep, [3, 0, 2], 256, 4096, seed=spare, spare=spare)


def test_a_row_does_not_depend_on_its_place(ep):
    """Equal rows of a tile, and the row alone, give equal bits: the parts are
    joined in one order wherever the row is."""
    a, a_scale, offsets, w, w_scale = operands([32], 512, 7168, 3)
    a = a.view(torch.uint8)[:1].repeat(32, 1).view(F8)
    a_scale = a_scale[:1].repeat(32, 1)
    out = ep.expert_matmul_fp8(a, a_scale, offsets, w, w_scale)
    assert torch.equal(out, out[:1].expand(32, -1))
    q, scale = ep.expert_gate_up_fp8(a, a_scale, offsets, w, w_scale)
    assert torch.equal(q.view(torch.uint8), q.view(torch.uint8)[:1].expand(32, -1))
    assert torch.equal(scale, scale[:1].expand(32, -1))


def test_values_that_are_not_finite_stay_in_their_row(ep):
    a, a_scale, offsets, w, w_scale = operands([9], 256, 7168, 8)
    clean = ep.expert_matmul_fp8(a, a_scale, offsets, w, w_scale)
    a_scale[4, 50] = float("inf")
    a_scale[7, 3] = float("nan")
    out = ep.expert_matmul_fp8(a, a_scale, offsets, w, w_scale)
    keep = [r for r in range(9) if r not in (4, 7)]
    assert torch.equal(out[keep], clean[keep])
    assert not bool(out[4].isfinite().any()) and bool(out[7].isnan().all())


def test_repeated_back_to_back_and_in_a_graph(ep):
    """Chained calls (each starts while the one before ends) keep their bits."""
    sets = [operands([2, 0, 1], 768, 4096, s) for s in range(3)]
    want = [ep.expert_matmul_fp8(*s) for s in sets]
    torch.cuda.synchronize()
    for _ in range(200):
        for s, x in zip(sets, want):
            got = ep.expert_matmul_fp8(*s)
    torch.cuda.synchronize()
    assert torch.equal(got, want[-1])
    outs = [torch.zeros_like(x) for x in want]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for _ in range(10):
            for s, o in zip(sets, outs):
                ep.ep_expert_matmul_fp8(*s, o)
    for _ in range(5):
        for o in outs:
            o.zero_()
        graph.replay()
    torch.cuda.synchronize()
    for o, x in zip(outs, want):
        assert torch.equal(o, x)


def test_no_rows_and_bad_offsets(ep):
    a, a_scale, offsets, w, w_scale = operands([4, 3], 256, 4096, 5)
    good = ep.expert_matmul_fp8(a, a_scale, offsets, w, w_scale)
    out = torch.full_like(good, 5.0)
    ep.ep_expert_matmul_fp8(a, a_scale, torch.zeros_like(offsets), w, w_scale, out)
    assert bool((out == 5.0).all())
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    bad = offsets.clone()
    bad[2] = 8  # one row more than there are
    ep.ep_expert_matmul_fp8(a, a_scale, bad, w, w_scale, out, status)
    assert ep.ep_get_status(status) == ep.EP_ERR_BAD_SLOT
    assert torch.equal(out[:4], good[:4]) and bool((out[4:] == 5.0).all())
    # offsets that claim rows twice: more tiles than clusters, reported, inside
    many = torch.tensor([0, 2, 0, 2, 0, 2, 0, 2, 2], dtype=torch.int32, device="cuda")
    a8, s8, _, w8, ws8 = operands([1, 1] + [0] * 6, 256, 4096, 6)
    guard = torch.full((3, 256), 5.0, dtype=torch.bfloat16, device="cuda")
    status.zero_()
    ep.ep_expert_matmul_fp8(a8, s8, many, w8, ws8, guard[:2], status)
    assert ep.ep_get_status(status) == ep.EP_ERR_BAD_SLOT
    assert bool((guard[2] == 5.0).all())


def test_beside_a_busy_device(ep):
    """Clusters wait for SMs that other streams' products hold, and finish."""
    big = operands([128] * 40, 1024, 1024, 2)
    small = operands([1, 0, 2], 512, 7168, 4)
    want, want_big = ep.expert_matmul_fp8(*small), ep.expert_matmul_fp8(*big)
    streams = [torch.cuda.Stream() for _ in range(3)]
    torch.cuda.synchronize()
    got = []
    for i in range(60):
        with torch.cuda.stream(streams[i % 3]):
            got.append((ep.expert_matmul_fp8(*big), ep.expert_matmul_fp8(*small)))
    torch.cuda.synchronize()
    for b, s in got:
        assert torch.equal(b, want_big) and torch.equal(s, want)


def test_in_an_sm_partition(ep):
    """A partition's SMs may not hold a cluster: whole tiles there, same bounds."""
    part, _, _, _ = ep.ep_sm_partition(24)
    torch.cuda.synchronize()
    with torch.cuda.stream(torch.cuda.ExternalStream(part)):
        check_matmul(ep, [1, 2], 256, 7168, seed=7)
        check_gate_up(ep, [1, 2], 256, 7168, seed=7)
    torch.cuda.synchronize()
