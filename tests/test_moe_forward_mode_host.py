"""Forward-mode derivatives, which no differentiable call here has: a tangent is refused,
never dropped, whether gradients are recorded or not (torch's own operators keep
tangents under no_grad). On the CPU, with stand-ins for the library's calls."""
import pytest
import torch
from torch.autograd import forward_ad

bf = torch.bfloat16


@pytest.fixture
def mods(monkeypatch):
    """(ep, moe) whose calls leave zeros."""
    from combine_movement_gb300 import build
    build.build()
    from combine_movement_gb300 import ep, moe
    monkeypatch.setattr(ep, "ep_linear", lambda x, w, y, *rest, **kind: y.zero_())
    return ep, moe


def linear_arguments():
    return {"x": torch.ones(4, 16, dtype=bf), "w": torch.ones(8, 16, dtype=bf),
            "bias": torch.ones(8), "residual": torch.ones(4, 8, dtype=bf)}


@pytest.mark.parametrize("recorded", [True, False])
@pytest.mark.parametrize("name", ["x", "w", "bias", "residual"])
def test_linear_refuses_a_tangent(mods, recorded, name):
    args = linear_arguments()
    with torch.set_grad_enabled(recorded), forward_ad.dual_level():
        args[name] = forward_ad.make_dual(args[name], torch.ones_like(args[name]))
        with pytest.raises(NotImplementedError):
            mods[1].linear(**args)


@pytest.mark.parametrize("recorded", [True, False])
def test_linear_without_a_tangent(mods, recorded):
    with torch.set_grad_enabled(recorded), forward_ad.dual_level():
        assert mods[1].linear(**linear_arguments()).shape == (4, 8)
    with torch.inference_mode():
        assert mods[1].linear(**linear_arguments()).shape == (4, 8)


# -- the 8-bit layer ------------------------------------------------------------

FORWARD_FP8 = ["x", "topk_w", "w_gate_up", "s_gate_up", "w_down", "s_down"]


@pytest.mark.parametrize("recorded", [True, False])
@pytest.mark.parametrize("name", ["x", "topk_w", "s_gate_up", "s_down"])
def test_forward_fp8_refuses_a_tangent(mods, monkeypatch, recorded, name):
    monkeypatch.setattr(mods[1], "_forward_fp8", lambda x, *rest: torch.zeros_like(x))
    args = {n: torch.ones(4, 4) for n in FORWARD_FP8}
    args["topk_idx"] = torch.zeros(4, 4, dtype=torch.int64)
    with torch.set_grad_enabled(recorded), forward_ad.dual_level():
        assert mods[1].forward_fp8(**args).shape == (4, 4)
        args[name] = forward_ad.make_dual(args[name], torch.ones(4, 4))
        with pytest.raises(NotImplementedError):
            mods[1].forward_fp8(**args)
