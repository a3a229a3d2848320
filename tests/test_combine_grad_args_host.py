"""Which arguments ep_combine_grad can do without (checked before any CUDA
call; addresses are made up and never used)."""
import pytest
import torch

A = 0x10000


@pytest.fixture(scope="module")
def ep():
    from combine_movement_gb300 import build
    build.build()
    from combine_movement_gb300 import ep as mod
    return mod


def call(ep, dy=A, e=A, R=16, slot=A, w=A, T=8, H=128, K=2, de=A, dw=A):
    return ep.lib.ep_combine_grad(dy, e, R, slot, w, T, H, K, de, dw, None, None)


@pytest.mark.parametrize("bad", [dict(e=None), dict(e=None, de=None), dict(de=None, dw=None),
                                 dict(e=None, de=None, dw=None), dict(e=A + 8, dw=None),
                                 dict(e=A + 8, de=None), dict(R=0, w=None, de=None, dw=None)])
def test_refused(ep, bad):
    assert call(ep, **bad) == ep.EP_ERR_INVALID


# (past the checks; what follows needs a GPU)
@pytest.mark.parametrize("good", [dict(e=None, dw=None), dict(de=None), dict(dw=None),
                                  dict(R=0, e=None, de=None, dw=None)])
@pytest.mark.skipif(torch.cuda.is_available(), reason="the addresses are made up")
def test_accepted(ep, good):
    assert call(ep, **good) == ep.EP_ERR_CUDA


def test_binding(ep):
    bf = torch.bfloat16
    dy, rows = torch.zeros((5, 128), dtype=bf), torch.zeros((10, 128), dtype=bf)
    slot, w = torch.zeros((5, 2), dtype=torch.int32), torch.zeros((5, 2))
    with pytest.raises(ValueError, match="CUDA tensor"):
        ep.ep_combine_grad(dy, None, slot, w, rows, None)
    with pytest.raises(ValueError, match="expert_out: expected a tensor"):
        ep.ep_combine_grad(dy, None, slot, w, None, w)
    with pytest.raises(ValueError, match="expected shape"):
        ep.ep_combine_grad(dy, None, slot, w, rows[:, :64], None)
