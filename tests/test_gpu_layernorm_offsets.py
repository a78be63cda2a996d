"""Layer norm's backward of rows whose offset is far above their spread, and of constant
rows: x - mean is taken before the scaling, so that nothing large cancels."""
import pytest
import torch

from block_common import assert_close
from top_routing_grouped_02_gb300 import moe

pytestmark = pytest.mark.gpu

BF, HF, FP = torch.bfloat16, torch.float16, torch.float32
EPS = 1e-5


def rows(T, d, ld, dt, seed):
    """Constant rows of several values, and rows of a few steps of the type around an offset."""
    g = torch.Generator().manual_seed(seed)
    base = torch.tensor([517.3, -1000.1, 3.7, 0.1, -20011.0, 0.0, 1.0], dtype=torch.float64)
    off = base[torch.arange(T) % len(base)].to(dt).double()
    step = torch.finfo(dt).eps * off.abs().clamp(min=0.5)
    x = off[:, None] + step[:, None] * torch.randint(-6, 7, (T, d), generator=g)
    x[::2] = off[::2, None]
    buf = torch.zeros(T, ld, dtype=dt)
    buf[:, :d] = x.to(dt)
    return buf.cuda()[:, :d]


def backward(x, dy, gamma, mean, rstd):
    """The formula in 64 bits on the statistics as given, and the terms of its errors."""
    x, dy, gamma, mean, rstd = (t.double().cpu() for t in (x, dy, gamma, mean, rstd))
    r = rstd[:, None]
    xh, g = (x - mean[:, None]) * r, dy * gamma
    gm, gx = g.mean(1, keepdim=True), (g * xh).mean(1, keepdim=True)
    dx = r * (g - gm - xh * gx)
    size = r * (g.abs() + g.abs().mean(1, keepdim=True) + xh.abs() * (g * xh).abs().mean(1, keepdim=True))
    return dx, size, (dy * xh).sum(0), (dy * xh).abs().sum(0), dy.sum(0), dy.abs().sum(0)


@pytest.mark.parametrize("dt", [BF, HF, FP])
@pytest.mark.parametrize("T,d,ld", [(70, 2048, 2048), (70, 2047, 2047), (33, 256, 256), (41, 200, 203), (40, 4099, 4099),
                                    (400, 1024, 1024)])
def test_backward(T, d, ld, dt):
    x = rows(T, d, ld, dt, T + d)
    g = torch.Generator().manual_seed(d)
    dy = torch.randn(T, d, generator=g).to(dt).cuda()
    gamma = (torch.randn(d, generator=g) * 0.3 + 1).cuda()
    xd = x.double()
    mean = xd.mean(1)
    rstd = 1 / torch.sqrt((xd - mean[:, None]).square().mean(1) + EPS)
    mean, rstd = mean.float(), rstd.float()
    dx, dgamma, dbeta = moe.moe_layernorm_backward(dy, x, gamma, mean, rstd)
    wx, size, wg, sg, wb, sb = backward(x, dy, gamma, mean, rstd)
    # xhat: two roundings; the row's sums: 16 terms in a pair's chain, one sum of the pair
    # and two trees of 5, their products and quotient; then four operations: below 48
    assert_close(dx, wx, size, 48.0, "dx")
    # at most T additions in chains and 32 in trees, xhat's two roundings and the product
    assert_close(dgamma, wg, sg, T + 36.0, "dgamma")
    assert_close(dbeta, wb, sb, T + 32.0, "dbeta")
