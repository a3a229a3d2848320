"""Refusals of ep_clear_unused_rows, before any CUDA call (made-up addresses)."""
import pytest
import torch

A = 0x10000


@pytest.fixture(scope="module")
def ep():
    from combine_movement_gb300 import build
    build.build()
    from combine_movement_gb300 import ep as mod
    return mod


def call(ep, rows=A, R=16, slot=A, T=8, H=128, K=2, st=None):
    return ep.lib.ep_clear_unused_rows(rows, R, slot, T, H, K, st, None)


@pytest.mark.parametrize("bad", [dict(rows=None), dict(slot=None), dict(rows=A + 8), dict(slot=A + 2),
                                 dict(st=A + 1), dict(R=-1), dict(T=-1), dict(H=0), dict(H=12),
                                 dict(K=0), dict(K=33), dict(T=0, rows=None)])
def test_invalid(ep, bad):
    assert call(ep, **bad) == ep.EP_ERR_INVALID


@pytest.mark.parametrize("big", [dict(T=1 << 31), dict(R=1 << 31), dict(H=1 << 31), dict(T=1 << 62)])
def test_sizes_beyond_the_limits(ep, big):
    assert call(ep, **big) == ep.EP_ERR_UNSUPPORTED


def test_nothing_to_do(ep):
    assert call(ep, rows=None, R=0) == ep.EP_OK
    assert call(ep, rows=None, slot=None, R=0, T=0) == ep.EP_OK


def test_binding(ep):
    rows, slot = torch.zeros((4, 64), dtype=torch.bfloat16), torch.zeros((2, 2), dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA tensor"):
        ep.ep_clear_unused_rows(rows, slot)
    with pytest.raises(ValueError, match="expected torch.int32"):
        ep.ep_clear_unused_rows(rows, slot.long())
    with pytest.raises(ValueError, match="contiguous"):
        ep.ep_clear_unused_rows(rows[:, :32], slot)
