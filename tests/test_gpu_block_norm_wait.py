"""The block norms' bounded waits: a row whose copies never come gives NaN, not what the ring
held, and the device goes on. (No fault: the wait of about a second runs out.)"""
import pytest
import torch

from block_common import matrix
from top_routing_grouped_02_gb300 import moe

pytestmark = pytest.mark.gpu
BF, FP = torch.bfloat16, torch.float32


def rows_apart(got, want, row):
    """`row` is NaN throughout; every other row is NaN throughout or as wanted."""
    got, want = (v if v.dim() == 2 else v[:, None] for v in (got, want))
    assert torch.isnan(got[row]).all()
    lost = torch.isnan(got).all(-1)
    assert torch.equal(got[~lost], want[~lost])
    assert int(lost.sum()) < len(got) // 2


@pytest.mark.parametrize("T,d,ld,dt,gate,norms,row", [
    (1500, 200, 200, BF, "full", (1, 1), 700), (700, 4096, 4096, BF, "row", (1, 1), 0), (700, 2048, 2048, FP, None, (1, 0), 699),
    (1400, 1001, 1003, BF, "full", (1, 1), 700), (1000, 7167, 7167, BF, "full", (0, 1), 40),
    (900, 12296, 12304, BF, "row", (1, 1), 899), (900, 12299, 12301, BF, "row", (1, 1), 8)])
def test_a_row_that_never_comes(T, d, ld, dt, gate, norms, row):
    g = torch.Generator().manual_seed(d)
    x, b, dy, du = (matrix(T, d, dt, g, ld) for _ in range(4))
    z = {None: None, "full": matrix(T, d, dt, g, ld), "row": matrix(T, 1, FP, g)[:, 0].contiguous()}[gate]
    kw = dict(gate=z, post_norm=bool(norms[0]), pre_norm=bool(norms[1]), stats=True)
    want = moe.moe_block_norm(x, b, **kw)
    moe.moe_selftest_layernorm_withhold(row)
    got = moe.moe_block_norm(x, b, **kw)
    torch.cuda.synchronize()
    for p, q in zip(got, want):
        assert (p is None) == (q is None)
        if p is not None:
            rows_apart(p, q, row)
    args = (dy, du if norms[1] else None, x, b, None, None, want[2], want[3])
    wb = moe.moe_block_norm_backward(*args, gate=z)
    moe.moe_selftest_layernorm_withhold(row)
    gb = moe.moe_block_norm_backward(*args, gate=z)
    torch.cuda.synchronize()
    for p, q in zip(gb[:3], wb[:3]):
        if q is not None:
            rows_apart(p, q, row)
    assert torch.isnan(gb[3]).all() and (gb[4] is None or torch.isnan(gb[4]).all())
    # the calls after it are as ever
    again = moe.moe_block_norm_backward(*args, gate=z)
    assert all(p is q is None or torch.equal(p, q) for p, q in zip(again, wb))
    u = moe.moe_rmsnorm(x)
    moe.moe_selftest_layernorm_withhold(row)
    rows_apart(moe.moe_rmsnorm(x), u, row)
    assert torch.equal(moe.moe_rmsnorm(x), u)
