"""Which kernel an RMS norm's backward takes: its rows come through the ring, as the block norms' do."""
import pytest
import torch

from block_common import matrix
from launches import kernels
from test_gpu_block_norm_wait import rows_apart
from top_routing_grouped_02_gb300 import moe

pytestmark = pytest.mark.gpu
BF, FP16, F32 = torch.bfloat16, torch.float16, torch.float32


@pytest.mark.parametrize("res", [False, True])
@pytest.mark.parametrize("dt", [BF, FP16])
def test_every_width_of_aligned_rows(dt, res):
    """16-bit rows, with and without the residual's gradient: no width takes the rows kernel."""
    T, side = 4, torch.cuda.Stream()
    x, dy, dres = (torch.zeros(T, 16384, dtype=dt, device="cuda") for _ in range(3))
    rstd = torch.ones(T, device="cuda")
    scratch = torch.empty(1 << 24, dtype=torch.uint8, device="cuda")

    def call(d):
        view = [v.view(-1)[:T * d].view(T, d) for v in (dy, x, dres)]
        return moe.moe_rmsnorm_backward(view[0], view[1], None, rstd, dres=view[2] if res else None, scratch=scratch, stream=side)

    side.wait_stream(torch.cuda.current_stream())
    call(64)
    slow = []
    for d in range(8, 16385, 8):
        names = [k[0] for k in kernels(lambda: call(d), side)]
        assert len(names) == 2
        if not any("backward_ring_kernel" in k for k in names):
            slow.append(d)
    assert not slow, f"{len(slow)} widths, {slow[0]} to {slow[-1]}"


@pytest.mark.parametrize("T,d,ld,dt,row", [
    (1500, 200, 200, BF, 700), (700, 4096, 4096, BF, 0), (700, 7168, 7168, FP16, 699), (900, 12296, 12304, BF, 899),
    (1400, 1001, 1003, BF, 700), (700, 2048, 2048, F32, 40)])
def test_a_row_that_never_comes(T, d, ld, dt, row):
    g = torch.Generator().manual_seed(d)
    x, dy, res = (matrix(T, d, dt, g, ld) for _ in range(3))
    _, rstd = moe.moe_rmsnorm(x, stats=True)
    for dres in (None, res):
        want = moe.moe_rmsnorm_backward(dy, x, None, rstd, dres=dres)
        moe.moe_selftest_layernorm_withhold(row)
        got = moe.moe_rmsnorm_backward(dy, x, None, rstd, dres=dres)
        torch.cuda.synchronize()
        rows_apart(got[0], want[0], row)
        assert torch.isnan(got[1]).all()
        again = moe.moe_rmsnorm_backward(dy, x, None, rstd, dres=dres)
        assert all(torch.equal(p, q) for p, q in zip(again, want))
