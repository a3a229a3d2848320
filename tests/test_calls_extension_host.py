"""The binding's extension on arguments of the wrong kind: every one comes back as an
error of the binding, none as a crash. On the CPU; no call gets as far as the
library."""
import pytest
import torch

bf, f32, i64 = torch.bfloat16, torch.float32, torch.int64


@pytest.fixture(scope="module")
def ep():
    from combine_movement_gb300 import build
    build.build()
    from combine_movement_gb300 import ep as mod
    return mod


class Odd:
    """Has what a tensor has, with other things in it."""
    dtype, shape = bf, (2, "8")

    def is_contiguous(self):
        raise RuntimeError("no")

    def get_device(self):
        return "cuda"

    def data_ptr(self):
        return -1


def calls(ep):
    z = lambda *s, dtype=bf: torch.zeros(s, dtype=dtype)
    l, i, w = z(4, 8), z(4, 2, dtype=i64), z(4, 2, dtype=f32)
    return [
        lambda v: ep._calls.route(v, i, w, None, 0, 1, 1, 0, True, 1.0, None),
        lambda v: ep._calls.route(l, v, w, None, 0, 1, 1, 0, True, 1.0, None),
        lambda v: ep._calls.route(l, i, v, None, 0, 1, 1, 0, True, 1.0, None),
        lambda v: ep._calls.route(l, i, w, v, 0, 1, 1, 0, True, 1.0, None),
        lambda v: ep._calls.route(l, i, w, None, v, 1, 1, 0, True, 1.0, None),
        lambda v: ep._calls.route(l, i, w, None, 0, 1, 1, 0, v, 1.0, None),
        lambda v: ep._calls.route(l, i, w, None, 0, 1, 1, 0, True, v, None),
        lambda v: ep._calls.route_grad(w, l, i, v, 0, True, 1.0, None, None),
        lambda v: ep._calls.linear(v, z(6, 8), z(4, 6), None, 0, None, None, None, None),
        lambda v: ep._calls.linear(l, z(6, 8), z(4, 6), None, 0, v, None, None, None),
        lambda v: ep._calls.linear(l, z(6, 8), z(4, 6), None, 0, None, None, v, None),
        lambda v: ep._calls.act_grad(v, None, z(4, 8), None, 0, None),
        lambda v: ep._calls.grad_input(z(4, 8), v, z(4, 8), None, None),
        lambda v: ep._calls.grad_weight(z(4, 8), z(4, 8), v, False, None, None),
    ]


@pytest.mark.parametrize("n", range(14))
@pytest.mark.parametrize("value", [None, 0, -1, 1 << 70, 2.5, "x", b"x", (), Odd(), object(),
                                   torch.zeros(3), torch.zeros(2, 2, 2), torch.zeros(4, 8, dtype=bf)])
def test_wrong_arguments_come_back(ep, n, value):
    assert calls(ep)[n](value) == -1


@pytest.mark.parametrize("name,count", [("route", 11), ("route_grad", 9), ("linear", 9), ("act_grad", 6),
                                        ("grad_input", 5), ("grad_weight", 6), ("bind", 12)])
def test_wrong_number_of_arguments(ep, name, count):
    for n in (0, count - 1, count + 1):
        with pytest.raises(TypeError):
            getattr(ep._calls, name)(*[None] * n)


def test_the_binding_says_what_is_wrong(ep):
    z = torch.zeros
    with pytest.raises(ValueError):
        ep.ep_route(z(4, 8), z(4, 2, dtype=i64), z(4, 2), groups="two")
    with pytest.raises(ValueError, match="activation"):
        ep.ep_linear(z(4, 8, dtype=bf), z(6, 8, dtype=bf), z(4, 6, dtype=bf), activation=None)
    with pytest.raises(ValueError, match="status"):
        ep.ep_linear(z(4, 8, dtype=bf), z(6, 8, dtype=bf), z(4, 6, dtype=bf), status=z(1, dtype=torch.int32))
