"""Where a projection's bias gradient is summed: beside the weight gradient, or by a kernel of its own."""
import pytest
import torch

from launches import kernels
from test_gpu_linear import BF, F32, inputs, unblocked
from top_routing_grouped_02_gb300 import moe

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T,k,n", [(40000, 256, 256), (16384, 1024, 512), (80000, 64, 64)])
def test_many_partial_rows_of_the_bias_gradient(T, k, n):
    """With many rows of partial sums the bias' gradient is a kernel of its own, beside dW too: one
    warp a CTA, which adds a column's partial rows one after the other, is not left behind with them
    when the products are done."""
    m = inputs((T, k, n, BF, F32, "silu", False))
    ws = moe.linear_workspace(T, k, n, train=True)
    side = torch.cuda.Stream()
    _, f = moe.moe_linear_train(m["x"], m["W"], m["bias"], act="silu", ws=ws)
    dA = m["dY"].double() * unblocked(f, T, n).double()
    want, terms = dA.sum(0), dA.abs().sum(0)
    db = moe.moe_linear_backward(m["dY"], m["x"], m["W"], f, bias_dtype=F32, ws=ws)[2]
    assert ((db.double() - want).abs() <= 2.0 ** -24 * want.abs() + T * 2.0 ** -23 * terms).all()
    side.wait_stream(torch.cuda.current_stream())
    count = [len(kernels(lambda: moe.moe_linear_backward(m["dY"], m["x"], m["W"], f, bias_dtype=b, ws=ws, stream=side), side))
             for b in (None, F32)]
    assert count[1] == count[0] + 1


def test_few_partial_rows_ride_with_the_weight_gradient():
    T, k, n = 777, 1000, 2728
    m = inputs((T, k, n, BF, F32, "gelu", False))
    ws, side = moe.linear_workspace(T, k, n, train=True), torch.cuda.Stream()
    _, f = moe.moe_linear_train(m["x"], m["W"], m["bias"], act="gelu", ws=ws)
    moe.moe_linear_backward(m["dY"], m["x"], m["W"], f, bias_dtype=F32, ws=ws)
    side.wait_stream(torch.cuda.current_stream())
    for b in (None, F32):
        assert len(kernels(lambda: moe.moe_linear_backward(m["dY"], m["x"], m["W"], f, bias_dtype=b, ws=ws, stream=side), side)) == 2
