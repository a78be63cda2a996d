"""Layer norm and its backward against the 64-bit definition on a GB300."""
import pytest
import torch

from block_common import assert_close, layernorm, layernorm_backward, matrix
from top_routing_grouped_02_gb300 import moe

pytestmark = pytest.mark.gpu

BF, HF, FP = torch.bfloat16, torch.float16, torch.float32
EPS = 1e-5
# (T, d, ld): one element, odd, unaligned strides, vector widths, several rows a
# block, rows of every warp count class, past the register kernels' width
SHAPES = [(1, 1, 1), (3, 2, 2), (5, 7, 9), (2, 8, 8), (33, 33, 33), (4, 64, 72), (9, 256, 256),
          (1000, 264, 264), (7, 1000, 1003), (257, 1023, 1023), (3, 1536, 1536), (700, 2048, 2048),
          (5, 4095, 4098), (2, 4096, 4096), (310, 4104, 4104), (3, 8191, 8191), (3, 8192, 8192),
          (2, 8193, 8200), (5, 12288, 12288),
          # several rows a group, past the ring's length
          (9000, 264, 264), (3000, 1000, 1024), (1500, 2048, 2048), (1300, 4104, 4104),
          (1000, 7168, 7168), (330, 12288, 12296), (2000, 999, 999)]
TYPES = [(BF, BF), (BF, FP), (HF, HF), (HF, FP), (FP, FP)]


def make(T, d, ld, dt, wt, seed=0):
    g = torch.Generator().manual_seed(1000 * seed + 7 * T + d)
    x = matrix(T, d, dt, g, ld, 2.0, 0.75)
    gamma = matrix(1, d, wt, g, None, 0.3, 1.0)[0]
    beta = matrix(1, d, wt, g, None, 0.3)[0]
    dy = matrix(T, d, dt, g, ld)
    dres = matrix(T, d, dt, g, ld)
    return x, gamma, beta, dy, dres


def check_forward(x, gamma, beta, y, mean, rstd, eps=EPS):
    d = x.shape[1]
    wy, wm, wr, xh = layernorm(x.cpu(), None if gamma is None else gamma.cpu(),
                               None if beta is None else beta.cpu(), eps)
    big = x.double().abs().amax(1, keepdim=True).cpu()
    # fp32 sums by a tree: each term passes at most 8 serial and 10 + 5 tree additions,
    # 32 in all with the division; a centred element inherits the mean's error, and the
    # deviations' sum relative errors of the same size
    c = 32.0
    assert_close(mean, wm[:, 0], big[:, 0], c, "mean")
    # rstd: relative error half of the variance's: the sum's c/2, and the mean's error
    # against the spread (first order in it only where the spread is that small)
    rel = c + c * (big * wr)[:, 0]
    assert_close(rstd, wr[:, 0], wr[:, 0] * rel, 1.0, "rstd")
    ga = torch.ones(d, dtype=torch.float64) if gamma is None else gamma.cpu().double()
    be = torch.zeros(d, dtype=torch.float64) if beta is None else beta.cpu().double()
    terms = (ga.abs() * (xh.abs() * (4 + rel[:, None]) + c * big * wr)) + 2 * be.abs()
    assert_close(y, wy, terms, 1.0, "y")


@pytest.mark.parametrize("dt,wt", TYPES)
@pytest.mark.parametrize("T,d,ld", SHAPES)
def test_forward(T, d, ld, dt, wt):
    x, gamma, beta, _, _ = make(T, d, ld, dt, wt)
    y, mean, rstd = moe.moe_layernorm(x, gamma, beta, EPS, stats=True)
    check_forward(x, gamma, beta, y, mean, rstd)
    assert torch.equal(moe.moe_layernorm(x, gamma, beta, EPS), y)


@pytest.mark.parametrize("dt,wt", TYPES)
@pytest.mark.parametrize("T,d,ld", SHAPES)
def test_backward(T, d, ld, dt, wt):
    x, gamma, beta, dy, dres = make(T, d, ld, dt, wt, 1)
    _, mean, rstd = moe.moe_layernorm(x, gamma, beta, EPS, stats=True)
    for res in (None, dres):
        dx, dgamma, dbeta = moe.moe_layernorm_backward(dy, x, gamma, mean, rstd, dres=res)
        check_backward(x, gamma, dy, res, dx, dgamma, dbeta)


def check_backward(x, gamma, dy, res, dx, dgamma, dbeta):
    T, d = x.shape
    xc, dyc = x.cpu(), dy.cpu()
    gc = None if gamma is None else gamma.cpu()
    wx, wg, wb = layernorm_backward(dyc, xc, gc, EPS, None if res is None else res.cpu())
    _, _, rstd, xh = layernorm(xc, None, None, EPS)
    c = 32.0
    big = xc.double().abs().amax(1, keepdim=True)
    # xhat's own error (its mean's, times rstd, and rstd's), as in the forward
    exh = xh.abs() * (4 + c + c * big * rstd) + c * big * rstd
    g = dyc.double() * (1.0 if gc is None else gc.double())
    gm, gx = g.abs().mean(1, keepdim=True), (g * xh).abs().mean(1, keepdim=True)
    egx = c * gx + (g.abs() * exh).mean(1, keepdim=True)
    err = rstd * ((g.abs() + gm + xh.abs() * gx) * (c + c * big * rstd) + xh.abs() * egx + exh * gx)
    if res is not None:
        err = err + 2 * (res.cpu().double().abs() + wx.abs())
    assert_close(dx, wx, err, 1.0, "dx")
    # sums over T rows in chains of T / (blocks * groups) terms and a tree of at
    # most 304 partials: at most T + 32 additions a term
    n = min(T, 4096) + 32
    assert_close(dgamma, wg, (dyc.double().abs() * (n * xh.abs() + exh)).sum(0), 1.0, "dgamma")
    assert_close(dbeta, wb, n * dyc.double().abs().sum(0), 1.0, "dbeta")


def test_without_weights():
    x, _, beta, dy, _ = make(37, 520, 520, BF, FP, 2)
    y, mean, rstd = moe.moe_layernorm(x, stats=True)
    check_forward(x, None, None, y, mean, rstd)
    check_forward(x, None, beta, *moe.moe_layernorm(x, None, beta, EPS, stats=True))
    dx, dgamma, dbeta = moe.moe_layernorm_backward(dy, x, None, mean, rstd, wdtype=BF)
    assert dgamma.dtype == BF
    check_backward(x, None, dy, None, dx, dgamma, dbeta)


def test_empty():
    x = torch.empty(0, 64, device="cuda", dtype=BF)
    gamma = torch.ones(64, device="cuda", dtype=BF)
    y, mean, rstd = moe.moe_layernorm(x, gamma, gamma, EPS, stats=True)
    assert y.shape == x.shape
    dx, dgamma, dbeta = moe.moe_layernorm_backward(x, x, gamma, mean, rstd)
    assert dx.shape == x.shape
    assert not dgamma.any() and not dbeta.any()


@pytest.mark.parametrize("dt", [BF, HF, FP])
def test_offset_far_above_spread(dt):
    # the variance is taken about the row's own mean: a constant row has spread 0
    # and a row of 1000 + small keeps its spread
    x = torch.full((3, 2048), 512.0, dtype=dt, device="cuda")
    x[1, ::2] += 1.0 if dt != BF else 4.0
    x[2] = 0
    y, mean, rstd = moe.moe_layernorm(x, None, None, EPS, stats=True)
    check_forward(x, None, None, y, mean, rstd)
    assert not y[0].any() and not y[2].any()


def test_nonfinite_rows_stay_apart():
    x, gamma, beta, _, _ = make(5, 512, 512, BF, BF, 3)
    want = moe.moe_layernorm(x, gamma, beta, EPS)
    x = x.clone()
    x[1, 3] = float("inf")
    x[3, 500] = float("nan")
    y = moe.moe_layernorm(x, gamma, beta, EPS)
    assert torch.equal(y[[0, 2, 4]], want[[0, 2, 4]])
    assert torch.isnan(y[1]).all() and torch.isnan(y[3]).all()


def test_in_place_and_other_stream():
    x, gamma, beta, dy, dres = make(301, 1024, 1024, BF, FP, 4)
    y, mean, rstd = moe.moe_layernorm(x, gamma, beta, EPS, stats=True)
    dx, dgamma, dbeta = moe.moe_layernorm_backward(dy, x, gamma, mean, rstd, dres=dres)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    x2, dy2 = x.clone(), dy.clone()
    s.wait_stream(torch.cuda.current_stream())
    got = moe.moe_layernorm_backward(dy2, x, gamma, mean, rstd, dres=dres, dx=dy2, stream=s)
    moe.moe_layernorm(x2, gamma, beta, EPS, y=x2, stream=s)
    s.synchronize()
    assert torch.equal(x2, y) and torch.equal(dy2, dx)
    assert torch.equal(got[1], dgamma) and torch.equal(got[2], dbeta)


@pytest.mark.parametrize("d,ld", [(300, 304), (333, 333), (2048, 2048), (8193, 8193), (12288, 12290)])
def test_gradients_over_their_operands(d, ld):
    # dx in the place of dy or of dres, on every kernel
    x, gamma, beta, dy, dres = make(40, d, ld, BF, FP, 7)
    _, mean, rstd = moe.moe_layernorm(x, gamma, beta, EPS, stats=True)
    want = moe.moe_layernorm_backward(dy, x, gamma, mean, rstd, dres=dres)
    for k in (0, 1):
        bufs = [torch.empty(40, ld, dtype=BF, device="cuda")[:, :d].copy_(t) for t in (dy, dres)]
        got = moe.moe_layernorm_backward(bufs[0], x, gamma, mean, rstd, dres=bufs[1], dx=bufs[k])
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_offsets_past_32_bits():
    T, d = 270000, 8192  # 2.2e9 elements
    x = torch.empty(T, d, dtype=BF, device="cuda").normal_(generator=torch.Generator("cuda").manual_seed(0))
    gamma = torch.ones(d, device="cuda")
    y, mean, rstd = moe.moe_layernorm(x, gamma, None, EPS, stats=True)
    tail = slice(T - 64, T)
    want = moe.moe_layernorm(x[tail], gamma, None, EPS, stats=True)
    assert all(torch.equal(a[tail], b) for a, b in zip((y, mean, rstd), want))
    dx = moe.moe_layernorm_backward(y, x, gamma, mean, rstd)[0]
    assert torch.equal(dx[tail], moe.moe_layernorm_backward(y[tail], x[tail], gamma, mean[tail], rstd[tail])[0])


def test_rows_of_a_higher_rank():
    x, gamma, beta, _, _ = make(24, 96, 96, FP, FP, 5)
    y, mean, _ = moe.moe_layernorm(x.view(2, 3, 4, 96), gamma, beta, EPS, stats=True)
    assert y.shape == (2, 3, 4, 96) and mean.shape == (2, 3, 4)
    assert torch.equal(y.view(24, 96), moe.moe_layernorm(x, gamma, beta, EPS))


def test_gradient_against_differences():
    # central differences of the 64-bit forward along random directions
    g = torch.Generator().manual_seed(9)
    x, dy = (torch.randn(6, 40, generator=g, dtype=torch.float64) for _ in range(2))
    gamma = torch.rand(40, generator=g, dtype=torch.float64) + 0.5
    xs, gs, ds = (t.float().cuda() for t in (x, gamma, dy))
    _, mean, rstd = moe.moe_layernorm(xs, gs, None, EPS, stats=True)
    dx, dgamma, _ = moe.moe_layernorm_backward(ds, xs, gs, mean, rstd)
    h = 1e-5
    for _ in range(5):
        u = torch.randn(6, 40, generator=g, dtype=torch.float64)
        f = [(layernorm(x + k * h * u, gamma, None, EPS)[0] * dy).sum() for k in (1, -1)]
        got = float((dx.double().cpu() * u).sum())
        # truncation h^2 and cancellation 1e-16 / h leave about 1e-9; fp32 results 1e-5
        assert abs(got - float(f[0] - f[1]) / (2 * h)) < 1e-4 * float(u.norm() * dx.double().norm())
        v = torch.randn(40, generator=g, dtype=torch.float64)
        f = [(layernorm(x, gamma + k * h * v, None, EPS)[0] * dy).sum() for k in (1, -1)]
        got = float((dgamma.double().cpu() * v).sum())
        assert abs(got - float(f[0] - f[1]) / (2 * h)) < 1e-4 * float(v.norm() * dgamma.double().norm())


def test_graph_replay():
    x, gamma, beta, dy, _ = make(64, 768, 768, BF, BF, 6)
    want = moe.moe_layernorm(x, gamma, beta, EPS, stats=True)
    wd = moe.moe_layernorm_backward(dy, x, gamma, want[1], want[2])
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    xin = torch.zeros_like(x)
    with torch.cuda.graph(graph):
        y, mean, rstd = moe.moe_layernorm(xin, gamma, beta, EPS, stats=True)
        grads = moe.moe_layernorm_backward(dy, xin, gamma, mean, rstd)
    xin.copy_(x)
    graph.replay()
    torch.cuda.synchronize()
    for a, b in zip((y, mean, rstd) + grads, want + wd):
        assert torch.equal(a, b)


@pytest.mark.parametrize("T,d,ld,dt,wt", [(800, 7167, 7167, BF, FP), (1400, 5001, 5003, HF, HF), (500, 8191, 8194, BF, BF),
                                          (1200, 3001, 3001, FP, FP), (900, 4093, 4093, FP, FP)])
def test_wide_unaligned_rows_many_a_group(T, d, ld, dt, wt):
    # rings of one stage a group, which is used again and again
    x, gamma, beta, dy, dres = make(T, d, ld, dt, wt, 5)
    y, mean, rstd = moe.moe_layernorm(x, gamma, beta, EPS, stats=True)
    check_forward(x, gamma, beta, y, mean, rstd)
    for res in (None, dres):
        dx, dgamma, dbeta = moe.moe_layernorm_backward(dy, x, gamma, mean, rstd, dres=res)
        check_backward(x, gamma, dy, res, dx, dgamma, dbeta)
        again = moe.moe_layernorm_backward(dy, x, gamma, mean, rstd, dres=res)
        assert all(torch.equal(a, b) for a, b in zip(again, (dx, dgamma, dbeta)))
