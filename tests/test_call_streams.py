"""Whose memory the allocating calls use: outputs and workspaces of a call on
a stream come from that stream's part of torch's allocator, and the current
stream is recorded for outputs. On the CPU, with stand-ins for torch's streams
and for the library's calls."""
import contextlib
import types

import pytest
import torch


class Stream:
    def __init__(self, handle):
        self.cuda_stream = handle


class Tensor:
    """What torch.empty gave: the stream it belongs to and those recorded."""

    def __init__(self, shape, dtype, owner):
        self.shape = tuple(shape) if isinstance(shape, (tuple, list)) else (shape,)
        self.dtype, self.owner, self.recorded = dtype, owner, []

    def record_stream(self, s):
        self.recorded.append(s.cuda_stream)


@pytest.fixture
def world(monkeypatch):
    """(ep, calls): the current stream is 5; `calls` gets, for each call of
    the C ABI, its name, its stream and the fresh tensors it was given."""
    from combine_movement_gb300 import build
    build.build()
    from combine_movement_gb300 import ep
    state = types.SimpleNamespace(current=Stream(5))

    @contextlib.contextmanager
    def on(s):
        before, state.current = state.current, s
        yield
        state.current = before

    def empty(*shape, dtype=None, device=None):
        shape = shape[0] if len(shape) == 1 else shape
        return Tensor(shape, dtype, state.current.cuda_stream)

    monkeypatch.setattr(torch.cuda, "Stream", Stream)
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda handle, device=None: Stream(handle))
    monkeypatch.setattr(torch.cuda, "default_stream", lambda device=None: Stream(0))
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: state.current)
    monkeypatch.setattr(torch.cuda, "stream", on)
    monkeypatch.setattr(torch, "empty", empty)
    monkeypatch.setattr(torch, "empty_like", lambda t: empty(tuple(t.shape), dtype=t.dtype))
    monkeypatch.setattr(ep, "ep_layout_workspace_bytes", lambda *a: 4096)
    calls = []
    for name in ("ep_get_dispatch_layout", "ep_dispatch", "ep_combine", "ep_dispatch_fp8",
                 "ep_combine_grad", "ep_dispatch_grad", "ep_expert_matmul_fp8",
                 "ep_expert_gate_up_fp8"):
        def call(*args, name=name):
            assert state.current.cuda_stream == 5
            calls.append((name, args[-1], [t for t in args if isinstance(t, Tensor)]))
        monkeypatch.setattr(ep, name, call)
    return ep, calls


def the_calls(ep):
    f8, bf, f32, i32 = torch.float8_e4m3fn, torch.bfloat16, torch.float32, torch.int32
    z = torch.zeros
    x, slot, w = z((5, 256), dtype=bf), z((5, 2), dtype=i32), z((5, 2))
    rows, idx = z((10, 256), dtype=bf), z((5, 2), dtype=torch.int64)
    a, s, off = z((10, 256), dtype=f8), z((10, 2), dtype=f32), z(4, dtype=i32)
    we, ws = z((3, 256, 256), dtype=f8), z((3, 2, 2), dtype=f32)
    return {
        "get_dispatch_layout": (4, lambda st: ep.get_dispatch_layout(idx, 3, stream=st)),
        "dispatch": (1, lambda st: ep.dispatch(x, slot, 10, stream=st)),
        "dispatch with weights": (3, lambda st: ep.dispatch(x, slot, 10, w, stream=st)),
        "combine": (1, lambda st: ep.combine(rows, slot, w, stream=st)),
        "dispatch_fp8": (2, lambda st: ep.dispatch_fp8(x, slot, 10, stream=st)),
        "dispatch_fp8 with weights": (4, lambda st: ep.dispatch_fp8(x, slot, 10, w, stream=st)),
        "combine_grad": (2, lambda st: ep.combine_grad(x, rows, slot, w, stream=st)),
        "dispatch_grad": (1, lambda st: ep.dispatch_grad(rows, slot, stream=st)),
        "expert_matmul_fp8": (1, lambda st: ep.expert_matmul_fp8(a, s, off, we, ws, stream=st)),
        "expert_gate_up_fp8": (2, lambda st: ep.expert_gate_up_fp8(a, s, off, we, ws, stream=st)),
    }


NAMES = ["get_dispatch_layout", "dispatch", "dispatch with weights", "combine", "dispatch_fp8",
         "dispatch_fp8 with weights", "combine_grad", "dispatch_grad", "expert_matmul_fp8",
         "expert_gate_up_fp8"]


@pytest.mark.parametrize("name", NAMES)
@pytest.mark.parametrize("given,owner", [(None, 5), (Stream(9), 9), (9, 9), (0, 0), (5, 5),
                                         (Stream(5), 5)])
def test_memory_belongs_to_the_calls_stream(world, name, given, owner):
    ep, calls = world
    count, call = the_calls(ep)[name]
    out = call(given)
    (_, stream, fresh), = calls
    assert stream is given and len(fresh) == count
    assert all(t.owner == owner for t in fresh)
    out = out if isinstance(out, tuple) else (out,)
    assert all(t.recorded == ([] if owner == 5 else [5]) for t in out)
    inner = [t for t in fresh if not any(t is o for o in out)]  # the layout's workspace
    assert len(inner) == (name == "get_dispatch_layout")
    assert all(t.recorded == [] for t in inner)
