"""Residual dropout of 16-bit rows that are even in length and start on words, but not on
vectors: two elements an access."""
import pytest
import torch

from block_common import assert_close, dropout_scale, keep_mask, matrix
from top_routing_grouped_02_gb300 import moe

pytestmark = pytest.mark.gpu
SEED, OFFSET = 0x123456789ABCDEF0, (1 << 33) + 7


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("T,d,ld,first", [(5, 300, 304, 0), (3, 1500, 1508, 0), (9, 7166, 7170, 0), (40, 2, 6, 0),
                                          (33, 14, 14, 2), (2, 254, 258, 2), (17, 256, 264, 4), (1, 1022, 1022, 6)])
def test_rows_of_words(T, d, ld, first, dt):
    # first: elements before the first row (4, 8 or 12 bytes past a vector)
    g = torch.Generator().manual_seed(T * 31 + d)

    def rows():
        return matrix(1, T * ld + first, dt, g)[0][first:].view(T, ld)[:, :d]

    x, res, dy = rows(), rows(), rows()
    keep = keep_mask(T * d, 0.3, SEED, OFFSET).view(T, d)
    scale = dropout_scale(0.3)

    def dropped(t):
        return torch.where(keep, t.double().cpu() * scale, 0.0)

    for r in (None, res):
        want = dropped(x) + (0.0 if r is None else r.double().cpu())
        y = moe.moe_dropout(x, 0.3, SEED, OFFSET, residual=r)
        # the scale's rounding to fp32, one fused multiply-add
        assert_close(y, want, want.abs() + x.double().cpu().abs() * scale, 2.0, "y")
        base = torch.zeros(T, d, dtype=dt) if r is None else r.cpu()
        assert torch.equal(y.cpu()[~keep], base[~keep])
        # in place, in a buffer whose other elements stay
        buf = torch.full((T * ld + first,), 7.0, dtype=dt, device="cuda")
        over = buf[first:].view(T, ld)[:, :d].copy_(x)
        assert torch.equal(moe.moe_dropout(over, 0.3, SEED, OFFSET, residual=r, y=over), y)
        assert int((buf == 7.0).sum()) - int((over == 7.0).sum()) == buf.numel() - T * d
    dx = moe.moe_dropout_backward(dy, 0.3, SEED, OFFSET)
    assert_close(dx, dropped(dy), dropped(dy).abs(), 2.0, "dx")
