"""Layer norm of rows that no ring in shared memory holds (16 bits: past 18984 elements
forward, 16384 backward; fp32: 14240 and 8192), in every direction and in place."""
import pytest
import torch

from block_common import assert_close, layernorm, matrix
from top_routing_grouped_02_gb300 import moe

pytestmark = pytest.mark.gpu
BF, HF, FP = torch.bfloat16, torch.float16, torch.float32
EPS = 1e-5
# a thread of 1024 adds at most 24 elements, two trees of 5 join them; products, the
# quotient and the final operations: below 48 roundings a term
C = 48.0
CASES = [(T, d, ld, dt, wt) for dt, wt in ((BF, BF), (BF, FP), (HF, FP), (FP, FP))
         for T, d, ld in ([(3, 14336, 14336), (5, 14337, 14340), (700, 14344, 14344)] if dt is FP else
                          [(3, 19008, 19008), (5, 19001, 19003), (700, 19008, 19016)])]


def buffers(T, d, ld, dt, wt):
    g = torch.Generator().manual_seed(T + d)
    x = matrix(T, d, dt, g, ld, 2.0, 0.75)
    gamma, beta = matrix(1, d, wt, g, None, 0.3, 1.0)[0], matrix(1, d, wt, g, None, 0.3)[0]
    return x, gamma, beta, matrix(T, d, dt, g, ld), matrix(T, d, dt, g, ld)


def like(t):
    """A copy in rows of the same stride."""
    return torch.empty(t.shape[0], t.stride(0), dtype=t.dtype, device=t.device)[:, :t.shape[1]].copy_(t)


@pytest.mark.parametrize("T,d,ld,dt,wt", CASES)
def test_forward(T, d, ld, dt, wt):
    x, gamma, beta, _, _ = buffers(T, d, ld, dt, wt)
    y, mean, rstd = moe.moe_layernorm(x, gamma, beta, EPS, stats=True)
    wy, wm, wr, xh = layernorm(x, gamma, beta, EPS)
    big = x.double().abs().amax(1, keepdim=True)
    assert_close(mean, wm[:, 0], big[:, 0], C, "mean")
    rel = C + C * (big * wr)  # rstd's: the sum's, and the mean's error against the spread
    assert_close(rstd, wr[:, 0], (wr * rel)[:, 0], 1.0, "rstd")
    ga, be = gamma.double().abs(), beta.double().abs()
    assert_close(y, wy, ga * (xh.abs() * (4 + rel) + C * big * wr) + 2 * be, 1.0, "y")
    over = like(x)
    assert torch.equal(moe.moe_layernorm(over, gamma, beta, EPS, y=over), y)


@pytest.mark.parametrize("T,d,ld,dt,wt", CASES)
def test_backward(T, d, ld, dt, wt):
    x, gamma, beta, dy, dres = buffers(T, d, ld, dt, wt)
    _, mean, rstd = moe.moe_layernorm(x, gamma, beta, EPS, stats=True)
    # the formula in 64 bits on the statistics that the call takes
    r = rstd.double()[:, None]
    xh, g = (x.double() - mean.double()[:, None]) * r, dy.double() * gamma.double()
    gx = g * xh
    want = r * (g - g.mean(1, keepdim=True) - xh * gx.mean(1, keepdim=True))
    size = r * (g.abs() + g.abs().mean(1, keepdim=True) + xh.abs() * gx.abs().mean(1, keepdim=True))
    dyx = dy.double() * xh
    for res in (None, dres):
        dx, dgamma, dbeta = moe.moe_layernorm_backward(dy, x, gamma, mean, rstd, dres=res)
        total = want if res is None else want + res.double()
        assert_close(dx, total, size + (0 if res is None else (res.double().abs() + total.abs()) / 24), C, "dx")
        assert dgamma.dtype == dbeta.dtype == wt
        assert_close(dgamma, dyx.sum(0), dyx.abs().sum(0), T + 36.0, "dgamma")
        assert_close(dbeta, dy.double().sum(0), dy.double().abs().sum(0), T + 32.0, "dbeta")
        for k in range(1 if res is None else 2):  # dx over dy, over dres
            a, b = like(dy), None if res is None else like(res)
            got = moe.moe_layernorm_backward(a, x, gamma, mean, rstd, dres=b, dx=(a, b)[k])
            assert all(torch.equal(p, q) for p, q in zip(got, (dx, dgamma, dbeta)))
        only = moe.moe_layernorm_backward(dy, x, gamma, mean, rstd, dres=res)
        assert all(torch.equal(p, q) for p, q in zip(only, (dx, dgamma, dbeta)))


@pytest.mark.parametrize("dt,d,ld", [(FP, 8193, 8200), (FP, 12288, 12290), (BF, 16390, 16390), (HF, 16384, 16384)])
def test_gradients_over_their_operands(dt, d, ld):
    # on both sides of the backward's ring
    x, gamma, beta, dy, dres = buffers(40, d, ld, dt, FP)
    _, mean, rstd = moe.moe_layernorm(x, gamma, beta, EPS, stats=True)
    want = moe.moe_layernorm_backward(dy, x, gamma, mean, rstd, dres=dres)
    for k in (0, 1):
        bufs = [like(dy), like(dres)]
        got = moe.moe_layernorm_backward(bufs[0], x, gamma, mean, rstd, dres=bufs[1], dx=bufs[k])
        assert all(torch.equal(p, q) for p, q in zip(got, want))
