"""The status word of the differentiable router and product: every call that may report
into it, forward or backward, is given the caller's. On the CPU, with stand-ins for the
library's calls that keep what they were given."""
import pytest
import torch

bf = torch.bfloat16


@pytest.fixture
def mods(monkeypatch):
    """(moe, seen): the status of each call by its name."""
    from combine_movement_gb300 import build
    build.build()
    from combine_movement_gb300 import ep, moe
    seen = {}

    def ep_linear(x, w, y, bias, activation, residual, z, status):
        seen["ep_linear"] = status
        y.zero_()

    def linear(x, w, bias, activation, residual, out_dtype, status):
        seen["linear"] = status
        return torch.zeros(x.shape[0], w.shape[0], dtype=out_dtype)

    def ep_linear_grad_input(dz, w, dx, status):
        seen["ep_linear_grad_input"] = status

    def ep_linear_grad_weight(dz, x, d_w, status):
        seen["ep_linear_grad_weight"] = status

    def route_grad(d, l, idx, score, renormalize, scale, status):
        seen["route_grad"] = status
        return torch.zeros_like(l)

    monkeypatch.setattr(ep, "ep_linear", ep_linear)
    monkeypatch.setattr(ep, "linear", linear)
    monkeypatch.setattr(ep, "ep_linear_grad_input", lambda dz, w, dx, status=None:
                        ep_linear_grad_input(dz, w, dx, status))
    monkeypatch.setattr(ep, "ep_linear_grad_weight", lambda dz, x, d_w, accumulate=False, status=None:
                        ep_linear_grad_weight(dz, x, d_w, status))
    monkeypatch.setattr(ep, "route", lambda l, k, *rest, **kind: (torch.zeros(l.shape[0], k, dtype=torch.int64),
                                                                  torch.ones(l.shape[0], k)))
    monkeypatch.setattr(ep, "route_grad", lambda d, l, idx, score="softmax", renormalize=True, scale=1.0,
                        status=None: route_grad(d, l, idx, score, renormalize, scale, status))
    return moe, seen


@pytest.mark.parametrize("given", [True, False])
def test_linear(mods, given):
    moe, seen = mods
    status = torch.zeros(1, dtype=torch.int32) if given else None
    x, w = torch.ones(4, 16, dtype=bf, requires_grad=True), torch.ones(8, 16, dtype=bf, requires_grad=True)
    moe.linear(x, w, status=status).sum().backward()
    assert set(seen) == {"ep_linear", "ep_linear_grad_input", "ep_linear_grad_weight"}
    with torch.no_grad():
        moe.linear(x, w, status=status)
    assert len(seen) == 4 and all(s is status for s in seen.values())


@pytest.mark.parametrize("given", [True, False])
def test_route(mods, given):
    moe, seen = mods
    status = torch.zeros(1, dtype=torch.int32) if given else None
    l = torch.zeros(4, 16, requires_grad=True)
    moe.route(l, 2, status=status)[1].sum().backward()
    assert set(seen) == {"route_grad"} and seen["route_grad"] is status


def test_a_status_that_is_cleared_before_the_backward_pass(mods):
    """A step's status is read and cleared between its calls."""
    moe, seen = mods
    status = torch.zeros(1, dtype=torch.int32)
    x = torch.ones(4, 16, dtype=bf, requires_grad=True)
    y = moe.linear(x, torch.ones(8, 16, dtype=bf), status=status)
    status.zero_()
    y.sum().backward()
    assert seen["ep_linear_grad_input"] is status
