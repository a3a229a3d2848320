"""The router's weights and their gradient where logits lie far apart: the rounding of a
logit's difference from the largest, half a unit of 2^-24 of up to 128, would be up
to 32 units of 2^-23 of e^difference.

Bounds. Weights: the header's 16 units of 2^-23 of their value, softmax weights that are
not renormalised E / 32 more; below 2^-125 they may be 0. The gradient: the 40 units and
E / 32 of test_gpu_route.py, for softmax that is not renormalised, whose gradient
reaches the experts that were not chosen, half of a logit's distance from the largest
more. A score that is 0 in place of up to 2^-125 takes as much of the magnitudes of g that
it is multiplied by, which are at most twice the token's largest.
"""
import pytest
import torch

from test_gpu_route import grad64, reference

pytestmark = pytest.mark.gpu
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


def wide(T, E, spread, shift, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn((T, E), generator=g) * spread + shift).to(dtype).cuda()


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("biased", [False, True])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("E,K,spread,shift", [(8, 8, 20, 0), (8, 8, 40, 0), (60, 32, 20, 0), (256, 32, 30, 0),
                                              (8, 8, 12, -60), (60, 32, 15, -100), (1000, 32, 25, -40)])
def test_weights(ep, score, renorm, biased, dtype, E, K, spread, shift):
    l = wide(300, E, spread, shift, dtype, E + spread)
    bias = torch.rand(E, generator=torch.Generator().manual_seed(1)).cuda() * 0.1 if biased else None
    idx, w = ep.route(l, K, bias, score, renormalize=renorm)
    ref_idx, ref = reference(l, K, bias, score, 1, 1, "max", renorm, 1.0)
    assert torch.equal(idx.cpu(), ref_idx)
    units = 16 + (0 if renorm else E / 32)
    err = (w.cpu().to(f64) - ref).abs()
    bad = (err > units * 2.0 ** -23 * ref) & ((ref >= 2.0 ** -125) | (err > 2.0 ** -125))
    assert not bool(bad.any()), (int(bad.sum()), float((err / ref)[bad].max()) * 2 ** 23)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("E,K,spread,shift", [(8, 8, 20, 0), (60, 32, 20, 0), (256, 32, 30, 0), (8, 8, 12, -60),
                                              (60, 32, 15, -100), (1000, 32, 25, -40)])
def test_gradient(ep, score, renorm, E, K, spread, shift):
    l = wide(300, E, spread, shift, torch.float32, E + spread)
    idx, _ = ep.route(l, K, None, score, renormalize=renorm)
    dw = torch.randn((300, K), generator=torch.Generator().manual_seed(E)).cuda()
    d = ep.route_grad(dw, l, idx, score, renorm)
    if score == "sigmoid" and renorm:
        # by the definition's last line: the scores' own ratios, which torch's
        # differentiation through their sum would lose at its 64 bits' end
        s = torch.sigmoid(l.cpu().to(f64)).gather(1, idx.cpu())
        p = s / s.sum(dim=1, keepdim=True)
        g = dw.cpu().to(f64)
        dot = (g * p).sum(dim=1, keepdim=True)
        want = torch.zeros(l.shape, dtype=f64).scatter_add_(1, idx.cpu(), p * (1 - s) * (g - dot))
        size = torch.zeros(l.shape, dtype=f64).scatter_add_(
            1, idx.cpu(), p * (g.abs() + (g.abs() * p).sum(dim=1, keepdim=True)))
    else:
        want, size = grad64(dw, l, idx, score, renorm, 1.0)
    units = 40 + E / 32
    if score == "softmax" and not renorm:
        l64 = l.cpu().to(f64)
        units = units + (l64.amax(dim=1, keepdim=True) - l64) / 2
    none = 2.0 ** -125 * 2 * dw.cpu().to(f64).abs().amax(dim=1, keepdim=True)
    bad = (d.cpu().to(f64) - want).abs() > units * 2.0 ** -23 * size + none
    assert not bool(bad.any()), int(bad.sum())
