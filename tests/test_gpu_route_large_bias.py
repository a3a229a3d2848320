"""Biases near fp32's largest number: a group's two largest then add up past its range,
where 64 bits still tell two groups apart. The choice equals the definition's."""
import pytest
import torch

from test_gpu_route import check

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
@pytest.mark.parametrize("sign", ["both", "up", "down"])
@pytest.mark.parametrize("E,groups,kept,K", [(64, 8, 4, 8), (128, 16, 5, 8), (256, 8, 3, 8), (256, 32, 9, 16),
                                             (60, 4, 2, 6), (512, 16, 4, 8)])
def test_sums_past_the_range(ep, score, sign, E, groups, kept, K):
    g = torch.Generator().manual_seed(E + groups)
    for _ in range(8):
        bias = torch.randn(E, generator=g).mul_(2e38).clamp_(-3.4e38, 3.4e38)
        bias = {"both": bias, "up": bias.abs(), "down": -bias.abs()}[sign]
        l = torch.randn((6, E), generator=g).cuda()
        check(ep, l, K, bias.cuda(), score, groups, kept, "top2")
        check(ep, l, K, bias.cuda(), score, groups, kept, "max")
