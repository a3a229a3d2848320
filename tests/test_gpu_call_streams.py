"""The allocating calls on another stream than the current one: results, and
whose memory they use."""
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


def calls(ep):
    g = torch.Generator(device="cuda").manual_seed(1)
    T, H, E, K = 300, 1024, 8, 4
    idx = torch.rand((T, E), generator=g, device="cuda").argsort(1)[:, :K].contiguous()
    x = torch.randn((T, H), generator=g, device="cuda").to(torch.bfloat16)
    w = torch.rand((T, K), generator=g, device="cuda")
    rows = torch.randn((T * K, H), generator=g, device="cuda").to(torch.bfloat16)
    weights = torch.randn((E, 512, H), generator=g, device="cuda").to(torch.float8_e4m3fn)
    scale = torch.rand((E, 4, 8), generator=g, device="cuda")
    _, offsets, slot = ep.get_dispatch_layout(idx, E)
    q, qs = ep.dispatch_fp8(x, slot, T * K)
    return {
        "layout": lambda s: ep.get_dispatch_layout(idx, E, stream=s),
        "dispatch": lambda s: ep.dispatch(x, slot, T * K, w, stream=s),
        "combine": lambda s: ep.combine(rows, slot, w, stream=s),
        "dispatch_fp8": lambda s: ep.dispatch_fp8(x, slot, T * K, w, stream=s),
        "combine_grad": lambda s: ep.combine_grad(x, rows, slot, w, stream=s),
        "dispatch_grad": lambda s: ep.dispatch_grad(rows, slot, stream=s),
        "matmul": lambda s: ep.expert_matmul_fp8(q, qs, offsets, weights, scale, stream=s),
        "gate_up": lambda s: ep.expert_gate_up_fp8(q, qs, offsets, weights, scale, stream=s),
    }


def tensors(out):
    return out if isinstance(out, tuple) else (out,)


@pytest.mark.parametrize("form", ["object", "handle", "partition", "default"])
def test_results_and_memory(ep, form):
    if form == "partition":
        side = torch.cuda.ExternalStream(ep.ep_sm_partition(24)[0])
    elif form == "default":
        side = torch.cuda.default_stream()
    else:
        side = torch.cuda.Stream()
    given = side.cuda_stream if form in ("handle", "default") else side
    here = torch.cuda.Stream() if form == "default" else torch.cuda.current_stream()
    cases = calls(ep)
    torch.cuda.synchronize()
    with torch.cuda.stream(here):
        for name, call in cases.items():
            want = [t.clone() for t in tensors(call(None))]
            here.synchronize()
            out = tensors(call(given))
            here.wait_stream(side)
            for a, b in zip(out, want):
                assert torch.equal(a.view(torch.uint8), b.view(torch.uint8)), name
            # dropped early, its memory is not the current stream's to hand out
            ptrs = {t.data_ptr() for t in out}
            shapes = [(t.shape, t.dtype) for t in out]
            del out, a
            again = [torch.empty(s, dtype=d, device="cuda") for s, d in shapes for _ in range(3)]
            assert ptrs.isdisjoint(t.data_ptr() for t in again), name
            torch.cuda.synchronize()
