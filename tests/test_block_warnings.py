"""A refusal of the sub-block calls reaches the caller also where torch has a warning to give
on the way. No GPU is needed: reading the address of a tensor that has no memory warns."""
import pytest
import torch
from torch._subclasses.fake_tensor import FakeTensorMode

from top_routing_grouped_02_gb300 import _build, moe


@pytest.fixture
def every_warning():
    before = torch.is_warn_always_enabled()
    torch.set_warn_always(True)
    yield
    torch.set_warn_always(before)


@pytest.mark.filterwarnings("always")
def test_refusal_after_a_warning(every_warning):
    _build.build()
    with FakeTensorMode():
        x, W1, W2 = (torch.empty(*s, dtype=torch.bfloat16, device="cuda:0") for s in ((4, 64), (64, 128), (128, 64)))
        ws = torch.empty(1 << 20, dtype=torch.uint8, device="cuda:0")
        other = W2.to(torch.float16)
    with pytest.warns(UserWarning, match="data pointer"):
        with pytest.raises(ValueError, match="W2 must be"):
            moe.moe_ffn(x, W1, W1, other, ws=ws)


@pytest.mark.filterwarnings("error")
def test_refusal_after_a_warning_that_raises(every_warning):
    # either may come through, but as itself
    _build.build()
    with FakeTensorMode():
        x, W1, W2 = (torch.empty(*s, dtype=torch.bfloat16, device="cuda:0") for s in ((4, 64), (64, 128), (64, 128)))
        ws = torch.empty(1 << 20, dtype=torch.uint8, device="cuda:0")
    with pytest.raises((ValueError, UserWarning), match="W2 must be|data pointer"):
        moe.moe_ffn(x, W1, W1, W2, ws=ws)
