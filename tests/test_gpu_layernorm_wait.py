"""Layer norm's bounded waits: a row whose copies never come gives NaN, not what the ring
held, and the device goes on. (No fault: the wait of about a second runs out.)"""
import pytest
import torch

from block_common import matrix
from top_routing_grouped_02_gb300 import moe

pytestmark = pytest.mark.gpu
BF, FP = torch.bfloat16, torch.float32


def rows_apart(got, want, row):
    """`row` is NaN throughout; every other row is NaN throughout or as wanted."""
    assert torch.isnan(got[row]).all()
    lost = torch.isnan(got).all(-1)
    assert torch.equal(got[~lost], want[~lost])
    assert int(lost.sum()) < len(got) // 2


@pytest.mark.parametrize("T,d,ld,dt,row", [(3000, 200, 200, BF, 1500), (700, 2048, 2048, BF, 0), (700, 4096, 4096, FP, 699),
                                           (1400, 1001, 1003, BF, 700), (1000, 7167, 7167, BF, 40)])
def test_a_row_that_never_comes(T, d, ld, dt, row):
    g = torch.Generator().manual_seed(d)
    x, dy, dres = (matrix(T, d, dt, g, ld) for _ in range(3))
    w = torch.ones(d, device="cuda")
    want = moe.moe_layernorm(x, w, None, stats=True)
    moe.moe_selftest_layernorm_withhold(row)
    got = moe.moe_layernorm(x, w, None, stats=True)
    torch.cuda.synchronize()
    rows_apart(got[0], want[0], row)
    assert torch.isnan(got[1][row]) and torch.isnan(got[2][row])
    for res in (None, dres):
        wb = moe.moe_layernorm_backward(dy, x, w, want[1], want[2], dres=res)
        moe.moe_selftest_layernorm_withhold(row)
        gb = moe.moe_layernorm_backward(dy, x, w, want[1], want[2], dres=res)
        torch.cuda.synchronize()
        rows_apart(gb[0], wb[0], row)
        assert torch.isnan(gb[1]).all() and torch.isnan(gb[2]).all()
        # the calls after it are as ever
        again = moe.moe_layernorm_backward(dy, x, w, want[1], want[2], dres=res)
        assert all(torch.equal(a, b) for a, b in zip(again, wb))
    assert all(torch.equal(a, b) for a, b in zip(moe.moe_layernorm(x, w, None, stats=True), want))
