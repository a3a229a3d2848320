"""Sizes that no call takes have no tiles (nothing here gets as far as a device)."""
import pytest
import torch


@pytest.fixture(scope="module")
def ep():
    from combine_movement_gb300 import build
    build.build()
    from combine_movement_gb300 import ep as mod
    return mod


@pytest.mark.parametrize("bad", [dict(product=3), dict(product=-1), dict(M=0), dict(N=0), dict(K=12), dict(K=0),
                                 dict(activation=5), dict(activation=-1), dict(out_type=2), dict(M=1 << 31),
                                 dict(M=(1 << 31) - 300, N=1 << 20), dict(product=1, activation=1),
                                 dict(product=2, activation=4), dict(product=1, out_type=1),
                                 dict(product=1, epilogue=1), dict(product=2, N=(1 << 31) - 300, K=1 << 20)])
def test_sizes_that_no_call_takes(ep, bad):
    a = dict(product=0, M=8, N=32, K=64, activation=0, out_type=0, epilogue=0)
    a.update(bad)
    assert ep.lib.ep_linear_tiles(*a.values(), None, None, None) == -1


@pytest.mark.parametrize("bad", [dict(product="act_grad"), dict(activation="tanh"), dict(out_dtype=torch.float16)])
def test_names(ep, bad):
    with pytest.raises(ValueError, match=next(iter(bad))):
        ep.ep_linear_tiles(**{**dict(product="linear", M=8, N=32, K=64), **bad})
