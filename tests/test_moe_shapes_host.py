"""The layer's calls refuse tensors whose sizes do not fit each other, before
anything is launched."""
import pytest
import torch


@pytest.fixture(scope="module")
def moe():
    from combine_movement_gb300 import build
    build.build()
    from combine_movement_gb300 import moe as mod
    return mod


bf, i32 = torch.bfloat16, torch.int32


@pytest.mark.parametrize("slot", [(4, 2), (6, 2), (10,), (5, 2, 1)])
def test_dispatch(moe, slot):
    with pytest.raises(ValueError, match="slot: expected shape"):
        moe.dispatch(torch.zeros((5, 64), dtype=bf), torch.zeros(slot, dtype=i32), 10)


@pytest.mark.parametrize("slot,w", [((5, 2), (5, 1)), ((5, 2), (4, 2)), ((5, 2), (10,)),
                                    ((5, 2), (5, 3)), ((10,), (10,))])
def test_combine(moe, slot, w):
    with pytest.raises(ValueError, match="expected shape"):
        moe.combine(torch.zeros((10, 64), dtype=bf), torch.zeros(slot, dtype=i32), torch.zeros(w))


@pytest.mark.parametrize("x,w", [((4, 256), (5, 2)), ((6, 256), (5, 2)), ((5, 256), (5, 1)),
                                 ((5, 256), (6, 2)), ((256,), (5, 2))])
def test_forward_fp8(moe, x, w):
    f8 = torch.float8_e4m3fn
    with pytest.raises(ValueError, match="expected shape"):
        moe.forward_fp8(torch.zeros(x, dtype=bf), torch.zeros((5, 2), dtype=torch.int64),
                        torch.zeros(w), torch.zeros((3, 256, 256), dtype=f8), torch.zeros((3, 2, 2)),
                        torch.zeros((3, 256, 128), dtype=f8), torch.zeros((3, 2, 1)))
