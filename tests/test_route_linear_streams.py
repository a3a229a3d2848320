"""Whose memory the router's and the dense products' allocating calls use: that of
the call's stream, recorded for the current one. On the CPU, with the stand-ins of
the movement's calls."""
import pytest
import torch

from test_call_streams import Stream, world  # noqa: F401  (a fixture)


@pytest.fixture
def calls_of(world, monkeypatch):  # noqa: F811
    ep, calls = world

    def record(name):
        def call(*args):
            calls.append((name, args[-1], [t for t in args if type(t).__name__ == "Tensor"
                                           and not isinstance(t, torch.Tensor)]))
        return call
    for name in ("ep_route", "ep_route_grad", "ep_linear"):
        monkeypatch.setattr(ep, name, record(name))
    return ep, calls


CALLS = {
    "route": (2, lambda ep, st: ep.route(torch.zeros(5, 16), 3, stream=st)),
    "route_grad": (1, lambda ep, st: ep.route_grad(torch.zeros(5, 3), torch.zeros(5, 16),
                                                   torch.zeros(5, 3, dtype=torch.int64), stream=st)),
    "linear": (1, lambda ep, st: ep.linear(torch.zeros(5, 16, dtype=torch.bfloat16),
                                           torch.zeros(8, 16, dtype=torch.bfloat16), stream=st)),
}


@pytest.mark.parametrize("name", sorted(CALLS))
@pytest.mark.parametrize("given,owner", [(None, 5), (Stream(9), 9), (9, 9), (0, 0), (5, 5)])
def test_memory_belongs_to_the_calls_stream(calls_of, name, given, owner):
    ep, calls = calls_of
    count, call = CALLS[name]
    out = call(ep, given)
    (_, stream, fresh), = calls
    assert stream is given and len(fresh) == count
    assert all(t.owner == owner for t in fresh)
    out = out if isinstance(out, tuple) else (out,)
    assert all(t.recorded == ([] if owner == 5 else [5]) for t in out)
