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


# -- tangents that meet a backward pass (forward mode over reverse) ------------------

def backward_through(out, leaf):
    """out's gradient carries a tangent, though nothing before out does."""
    factor = forward_ad.make_dual(torch.ones_like(out), torch.ones_like(out))
    return torch.autograd.grad((out * factor).sum(), leaf)


@pytest.fixture
def movement(mods, monkeypatch):
    """moe, with stand-ins for the movement's and the router's calls too."""
    ep, moe = mods
    monkeypatch.setattr(ep, "dispatch", lambda x, slot, r: torch.zeros(r, x.shape[1], dtype=x.dtype))
    monkeypatch.setattr(ep, "dispatch_grad", lambda d, slot: torch.zeros(4, d.shape[1], dtype=d.dtype))
    monkeypatch.setattr(ep, "combine", lambda rows, slot, w: torch.zeros(4, rows.shape[1], dtype=rows.dtype))
    monkeypatch.setattr(ep, "route", lambda l, k, *rest, **kind: (torch.zeros(4, k, dtype=torch.int64),
                                                                  torch.ones(4, k)))
    monkeypatch.setattr(ep, "route_grad", lambda d, l, idx, *rest, **kind: torch.zeros_like(l))
    for name in ("ep_clear_unused_rows", "ep_combine_grad", "ep_linear_act_grad", "ep_linear_grad_input",
                 "ep_linear_grad_weight"):
        monkeypatch.setattr(ep, name, lambda *args, **kind: None)
    return moe


SLOT = torch.zeros(4, 2, dtype=torch.int32)
THROUGH = {
    "dispatch": (lambda moe, leaf: moe.dispatch(leaf, SLOT, 8), (4, 16), bf),
    "combine": (lambda moe, leaf: moe.combine(leaf, SLOT, torch.ones(4, 2)), (8, 16), bf),
    "linear": (lambda moe, leaf: moe.linear(leaf, torch.ones(8, 16, dtype=bf)), (4, 16), bf),
    "route": (lambda moe, leaf: moe.route(leaf, 2)[1], (4, 16), torch.float32),
}


@pytest.mark.parametrize("name", sorted(THROUGH))
def test_a_backward_pass_refuses_a_tangent(movement, name):
    call, shape, dtype = THROUGH[name]
    leaf = torch.ones(shape, dtype=dtype, requires_grad=True)
    with forward_ad.dual_level():
        out = call(movement, leaf)
        torch.autograd.grad(out.sum(), leaf, retain_graph=True)
        with pytest.raises((NotImplementedError, RuntimeError), match="forward"):
            backward_through(out, leaf)


def test_a_residual_keeps_its_tangent(movement):
    """Its gradient is the result's own."""
    leaf = torch.ones(4, 16, dtype=bf, requires_grad=True)
    with forward_ad.dual_level():
        out = movement.linear(torch.ones(4, 8, dtype=bf), torch.ones(16, 8, dtype=bf), residual=leaf)
        g, = backward_through(out, leaf)
        assert torch.equal(forward_ad.unpack_dual(g).tangent, torch.ones_like(leaf))
