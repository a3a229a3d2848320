"""ep_clear_unused_rows: zeros where no entry maps to, nothing else changed."""
import pytest
import torch

pytestmark = pytest.mark.gpu


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


def slots(T, K, rows, mask, seed):
    """slot [T, K]: unmasked entries on distinct rows, anywhere in the buffer."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    on = torch.rand((T, K), generator=g, device="cuda") >= mask
    n = min(int(on.sum()), rows)
    place = on.reshape(-1).nonzero()[:n, 0]
    slot = torch.full((T * K,), -1, dtype=torch.int32, device="cuda")
    slot[place] = torch.randperm(rows, generator=g, device="cuda")[:n].to(torch.int32)
    return slot.view(T, K)


def check(ep, slot, R, H, num_sms=0):
    # one guard row on either side
    buf = torch.full((R + 2, H), float("nan"), dtype=torch.bfloat16, device="cuda")
    used = torch.zeros(R, dtype=torch.bool, device="cuda")
    used[slot[slot >= 0].long()] = True
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    ep.ep_set_num_sms(num_sms)
    ep.ep_clear_unused_rows(buf[1:-1], slot, status)
    ep.ep_set_num_sms(0)
    assert ep.ep_get_status(status) == ep.EP_OK
    rows = buf[1:-1]
    assert bool((rows[~used] == 0).all()) and bool(rows[used].isnan().all())
    assert bool(buf[0].isnan().all()) and bool(buf[-1].isnan().all())


@pytest.mark.parametrize("T,K,R,H", [
    (1, 1, 1, 8), (1, 8, 8, 7168), (1, 1, 5, 16), (37, 3, 111, 40), (37, 3, 200, 248), (100, 4, 400, 256),
    (999, 8, 8000, 264), (4096, 8, 32768, 1024), (3000, 6, 20011, 2048), (2, 32, 4097, 1000)])
@pytest.mark.parametrize("mask", [0.0, 0.3, 1.1])
def test_sizes_and_masks(ep, T, K, R, H, mask):
    check(ep, slots(T, K, R, mask, T + R), R, H)


@pytest.mark.parametrize("num_sms", [1, 2, 3, 24, 151])
def test_sm_budget(ep, num_sms):
    check(ep, slots(500, 4, 2100, 0.2, 1), 2100, 512, num_sms)


def test_more_rows_than_a_map_holds(ep):
    """One CTA's bit map holds 983040 rows; these take it three times."""
    check(ep, slots(70000, 8, 2100000, 0.1, 2), 2100000, 8, num_sms=1)
    check(ep, slots(70000, 8, 2100000, 0.1, 2), 2100000, 8)


def test_no_tokens_and_no_rows(ep):
    slot = torch.zeros((0, 4), dtype=torch.int32, device="cuda")
    rows = torch.full((70, 64), 9.0, dtype=torch.bfloat16, device="cuda")
    ep.ep_clear_unused_rows(rows, slot)
    assert bool((rows == 0).all())
    ep.ep_clear_unused_rows(rows[:0], torch.full((3, 2), -1, dtype=torch.int32, device="cuda"))


def test_slots_past_the_buffer_are_reported(ep):
    slot = torch.tensor([[0, 9], [3, 2147483647], [10, -1]], dtype=torch.int32, device="cuda")
    rows = torch.full((10, 64), 9.0, dtype=torch.bfloat16, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    ep.ep_clear_unused_rows(rows, slot, status)
    assert ep.ep_get_status(status) == ep.EP_ERR_BAD_SLOT
    keep = torch.zeros(10, dtype=torch.bool, device="cuda")
    keep[[0, 9, 3]] = True
    assert bool((rows[keep] == 9).all()) and bool((rows[~keep] == 0).all())


def test_after_dispatch_in_a_graph_and_in_a_partition(ep):
    T, K, R, H = 700, 4, 3000, 1024
    slot = slots(T, K, R, 0.2, 5)
    x = torch.randn((T, H), device="cuda").to(torch.bfloat16)
    want = torch.zeros((R, H), dtype=torch.bfloat16, device="cuda")
    ep.ep_dispatch(x, slot, want)
    got = torch.full_like(want, float("nan"))
    side = torch.cuda.ExternalStream(ep.ep_sm_partition(24)[0])
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        ep.ep_dispatch(x, slot, got)
        ep.ep_clear_unused_rows(got, slot)
    torch.cuda.synchronize()
    assert torch.equal(got, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for _ in range(5):
            ep.ep_dispatch(x, slot, got)
            ep.ep_clear_unused_rows(got, slot)
    for _ in range(3):
        got.fill_(float("nan"))
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(got, want)
