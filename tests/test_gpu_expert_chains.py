"""Chained products of tiles that clusters share: every result of a long chain
keeps its bits, not the last alone."""
import pytest
import torch

from test_gpu_expert_fp8 import operands

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


def test_every_result_of_a_chain(ep):
    sets = [operands(counts, 768, 4096, s) for s, counts in enumerate([[2, 0, 1], [0, 5, 0], [1, 1, 30]])]
    want = [(ep.expert_matmul_fp8(*s), *ep.expert_gate_up_fp8(*s)) for s in sets]
    torch.cuda.synchronize()
    bits = [tuple(t.view(torch.uint8) for t in x) for x in want]
    got = [(i, ep.expert_matmul_fp8(*sets[i]), *ep.expert_gate_up_fp8(*sets[i]))
           for _ in range(200) for i in range(3)]
    torch.cuda.synchronize()
    for i, *x in got:
        assert all(torch.equal(t.view(torch.uint8), b) for t, b in zip(x, bits[i]))
