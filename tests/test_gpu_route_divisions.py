"""Weights of equal logits: exponentials and sums are whole numbers (sigmoid: halves), so
that the one division is all that is rounded, and has to be to the nearest."""
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


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_of_the_chosen(ep, score):
    for K in range(1, 33):
        _, w = ep.route(torch.zeros(3, 40, device="cuda"), K, None, score)
        assert torch.equal(w.cpu(), (torch.ones(3, K) / K)), K


def test_of_all(ep):
    for E in list(range(1, 70)) + [100, 255, 500, 1001]:
        _, w = ep.route(torch.full((3, E), -7.0, device="cuda"), 1, None, "softmax", renormalize=False)
        assert torch.equal(w.cpu(), (torch.ones(3, 1) / E)), E
