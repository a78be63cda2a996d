"""Arguments of the sub-block calls that are no truth value: the argument's own error comes
through, and nothing is launched."""
import pytest
import torch

from top_routing_grouped_02_gb300 import moe

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


def test_flags_without_a_truth_value():
    x = torch.randn(4, 64, device="cuda").to(BF)
    W1, W2 = torch.randn(64, 128, device="cuda").to(BF), torch.randn(128, 64, device="cuda").to(BF)
    neither = torch.ones(2)  # "Boolean value of Tensor with more than one value is ambiguous"
    saved = moe.moe_ffn_train(x, W1, W1, W2)[1:]
    for call in (lambda: moe.moe_layernorm(x, stats=neither),
                 lambda: moe.moe_ffn_backward(x, x, W1, W1, W2, *saved, need_dx=neither),
                 lambda: moe.moe_ffn_backward(x, x, W1, W1, W2, *saved, need_dw=neither)):
        with pytest.raises(RuntimeError, match="ambiguous"):
            call()
    assert moe.moe_layernorm(x).shape == x.shape
