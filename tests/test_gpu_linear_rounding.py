"""Projections' gradients against the products of the operands that the kernels take."""
import pytest
import torch

from block_common import HALF, TINY
from linear_common import E32
from test_gpu_linear import BF, F32, FP16, inputs, unblocked
from top_routing_grouped_02_gb300 import moe

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("case", [
    (777, 1000, 2728, BF, F32, "gelu", True), (1030, 2048, 200, FP16, FP16, "silu", True), (300, 520, 264, BF, BF, "silu", True),
    (2100, 136, 8, BF, BF, None, True), (17, 72, 40, FP16, None, "gelu", False)], ids=str)
def test_products_of_the_rounded_gradient(case):
    """dA = dY F in fp32, rounded once to the operands' type, is all that dX and dW lose: they are
    that dA's products, summed in fp32 (each of K products off by at most 2^-23 of the absolute
    terms) and rounded once. And they repeat themselves."""
    T, k, n, dt, bt, act, _ = case
    m = inputs(case)
    ws = moe.linear_workspace(T, k, n, train=True)
    _, f = moe.moe_linear_train(m["x"], m["W"], m["bias"], act=act, residual=m["res"], ws=ws)
    dA = m["dY"] if f is None else (m["dY"].float() * unblocked(f, T, n)).to(dt)
    dX, dW, _ = moe.moe_linear_backward(m["dY"], m["x"], m["W"], f, bias_dtype=bt, ws=ws)
    A, x, W = (v.double().cpu() for v in (dA, m["x"], m["W"]))
    for got, a, b, terms in ((dX, A, W.T, n), (dW, x.T, A, T)):
        want, slack = a @ b, terms * E32 * (a.abs() @ b.abs())
        err = (got.double().cpu() - want).abs()
        assert (err <= HALF[dt] * (want.abs() + slack) + slack + TINY[dt]).all()
    for _ in range(3):
        again = moe.moe_linear_backward(m["dY"], m["x"], m["W"], f, bias_dtype=bt, ws=ws)
        assert torch.equal(again[0], dX) and torch.equal(again[1], dW)
