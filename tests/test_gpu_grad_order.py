"""ep_combine_grad gives the same bits for the same inputs and SM budget on
every stream, an SM partition's among them: how many warps share an entry, and
so the order of its sum, goes by the budget alone."""
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
    return mod


# whole GPU: eight, four, two warps and one to an entry
@pytest.mark.parametrize("T,K,H", [(100, 2, 8192), (25, 8, 16384), (250, 4, 4096), (300, 8, 2048),
                                   (1000, 4, 7168)])
def test_in_an_sm_partition(ep, T, K, H):
    g = torch.Generator(device="cuda").manual_seed(T)
    dy = torch.randn((T, H), generator=g, device="cuda").to(torch.bfloat16)
    rows = torch.randn((T * K, H), generator=g, device="cuda").to(torch.bfloat16)
    slot = torch.randperm(T * K, generator=g, device="cuda").to(torch.int32).view(T, K)
    w = torch.rand((T, K), generator=g, device="cuda")
    want = ep.combine_grad(dy, rows, slot, w)
    part, rest, _, _ = ep.ep_sm_partition(24)
    torch.cuda.synchronize()
    for stream in (part, rest):
        with torch.cuda.stream(torch.cuda.ExternalStream(stream)):
            d_rows, d_w = ep.combine_grad(dy, rows, slot, w)
        torch.cuda.synchronize()
        assert torch.equal(d_rows, want[0]) and torch.equal(d_w, want[1])
