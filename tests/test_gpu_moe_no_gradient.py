"""The 8-bit layer has no gradient: its result says so where one is asked for,
instead of taking no part in the graph."""
import pytest
import torch

from combine_movement_gb300 import workloads as W

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def mods():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    torch.cuda.set_device(0)
    from combine_movement_gb300 import build
    build.build()
    from combine_movement_gb300 import ep, moe
    return ep, moe


@pytest.fixture(scope="module")
def layer(mods):
    _, moe = mods
    inp = W.make_inputs(W.Workload("layer", T=20, H=256, E=4, K=2, seed=1))
    g = torch.Generator(device="cuda").manual_seed(2)
    gate_up = torch.randn((4, 256, 256), generator=g, device="cuda") / 16
    down = torch.randn((4, 256, 128), generator=g, device="cuda") / 16
    args = [inp.x.cuda(), inp.topk_idx.cuda(), inp.topk_w.cuda(), *moe.quantize_weights(gate_up),
            *moe.quantize_weights(down)]
    return args, moe.forward_fp8(*args)


@pytest.mark.parametrize("which", [0, 2, 4, 6])  # x, topk_w, the weights' scales
def test_a_backward_pass_is_refused(mods, layer, which):
    _, moe = mods
    args, want = layer
    args = list(args)
    args[which] = args[which].clone().requires_grad_()
    y = moe.forward_fp8(*args)
    assert torch.equal(y.detach(), want)
    other = torch.ones(1, device="cuda", requires_grad=True)  # keeps the loss in a graph
    with pytest.raises(RuntimeError, match="forward_fp8 has no gradient"):
        (y.float().sum() + other.sum()).backward()


def test_without_gradients_nothing_is_asked(mods, layer):
    _, moe = mods
    args, want = layer
    args = list(args)
    args[0] = args[0].clone().requires_grad_()
    with torch.no_grad():
        y = moe.forward_fp8(*args)
    assert not y.requires_grad and torch.equal(y, want)
    assert not want.requires_grad
