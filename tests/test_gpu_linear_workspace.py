"""Projections onto the residual, in workspaces made for more tokens."""
import pytest
import torch

from test_gpu_linear import BF, F32, FP16, inputs
from top_routing_grouped_02_gb300 import moe

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("case", [
    (1, 128, 4096, BF, F32, "silu", True), (16, 1000, 2728, FP16, F32, "gelu", True), (33, 2048, 1032, BF, F32, None, True),
    (777, 1000, 2728, BF, F32, "gelu", True)], ids=str)
def test_onto_the_residual_in_a_workspace_of_more_tokens(case):
    T, k, n, act = *case[:3], case[5]
    m = inputs(case)
    want = moe.moe_linear(m["x"], m["W"], m["bias"], act=act, residual=m["res"])
    ws = moe.linear_workspace(T + 500, k, n, train=True)
    for _ in range(2):
        res = m["res"].clone()
        got = moe.moe_linear(m["x"], m["W"], m["bias"], act=act, residual=res, Y=res, ws=ws)
        assert got.data_ptr() == res.data_ptr() and torch.equal(got, want)
    assert moe.moe_sync_check(ws) == (0, 0)
