"""Residual dropout from the counter-based generator, on a GB300."""
import pytest
import torch

from block_common import assert_close, dropout_scale, keep_mask, matrix
from top_routing_grouped_02_gb300 import moe

pytestmark = pytest.mark.gpu

BF, HF, FP = torch.bfloat16, torch.float16, torch.float32
SEED, OFFSET = 0xDEADBEEF12345678, (3 << 40) + 5
SHAPES = [(1, 1, 1), (1, 7, 7), (3, 8, 8), (5, 13, 13), (5, 13, 16), (2, 256, 264), (17, 40, 48),
          (3, 300, 303), (11, 31, 31), (1, 4099, 4099), (64, 96, 96), (9, 5, 7)]


def want_dropout(x, p, res=None, seed=SEED, offset=OFFSET):
    T, d = x.shape
    keep = keep_mask(T * d, p, seed, offset).view(T, d)
    y = torch.where(keep, x.double().cpu() * dropout_scale(p), 0.0)
    return (y if res is None else y + res.double().cpu()), keep


@pytest.mark.parametrize("dt", [BF, HF, FP])
@pytest.mark.parametrize("p", [0.1, 0.5])
@pytest.mark.parametrize("T,d,ld", SHAPES)
def test_dropout(T, d, ld, p, dt):
    g = torch.Generator().manual_seed(T * 31 + d)
    x, res, dy = (matrix(T, d, dt, g, ld) for _ in range(3))
    for r in (None, res):
        y = moe.moe_dropout(x, p, SEED, OFFSET, residual=r)
        want, keep = want_dropout(x, p, r)
        # scale rounded to fp32, one fused multiply-add
        terms = want.abs() + x.double().cpu().abs() * dropout_scale(p)
        assert_close(y, want, terms, 2.0, "y")
        base = torch.zeros_like(x) if r is None else r
        assert torch.equal(y.cpu()[~keep], base.cpu()[~keep])
    dx = moe.moe_dropout_backward(dy, p, SEED, OFFSET)
    assert_close(dx, want_dropout(dy, p)[0], want_dropout(dy, p)[0].abs(), 2.0, "dx")


def test_mask_does_not_depend_on_type_or_layout():
    ones = torch.ones(40, 72, device="cuda")
    ref = moe.moe_dropout(ones, 0.3, 7, 9) != 0
    for dt in (BF, HF, FP):
        for ld in (72, 73, 80):
            x = torch.ones(40, ld, device="cuda", dtype=dt)[:, :72]
            assert torch.equal(moe.moe_dropout(x, 0.3, 7, 9) != 0, ref)
    shifted = torch.ones(40 * 72 + 1, device="cuda", dtype=BF)[1:].view(40, 72)
    assert torch.equal(moe.moe_dropout(shifted, 0.3, 7, 9) != 0, ref)


def test_edges_of_p():
    g = torch.Generator().manual_seed(1)
    x, res = matrix(33, 65, FP, g), matrix(33, 65, FP, g)
    assert torch.equal(moe.moe_dropout(x, 0.0, 1, 2), x)
    assert torch.equal(moe.moe_dropout(x, 1.0, 1, 2, residual=res), res)
    assert not moe.moe_dropout(x, 1.0, 1, 2).any()
    assert moe.moe_dropout(x[:0], 0.5, 1).shape == (0, 65)
    # the smallest and largest thresholds
    for p in (2.0 ** -16, 1 - 2.0 ** -16):
        want, keep = want_dropout(x, p, seed=1, offset=2)
        assert torch.equal((moe.moe_dropout(x, p, 1, 2) != 0).cpu(), keep & (x.cpu() != 0))


def test_dropped_elements_are_not_read_into_the_result():
    keep = keep_mask(4096, 0.5, 3, 4).view(64, 64)
    x = torch.where(keep, 1.0, float("nan")).to(BF).cuda()
    x[~keep.cuda()] = float("inf")
    y = moe.moe_dropout(x, 0.5, 3, 4, residual=torch.ones(64, 64, device="cuda", dtype=BF))
    assert torch.equal(y.cpu(), torch.where(keep, 3.0, 1.0).to(BF))


def test_statistics():
    # 2^22 draws: the count of kept is within 5 standard deviations, and so are the
    # pair counts of neighbours and of elements in consecutive blocks and offsets
    n, p = 1 << 22, 0.25
    ones = torch.ones(1, n, device="cuda")
    a = (moe.moe_dropout(ones, p, 11, 0) != 0)[0].double()
    b = (moe.moe_dropout(ones, p, 11, 1) != 0)[0].double()
    q = 1 - p
    dev = 5 * (q * p * n) ** 0.5
    assert abs(float(a.sum()) - q * n) < dev and abs(float(b.sum()) - q * n) < dev
    pair = 5 * (q * q * (1 - q * q) * n) ** 0.5 * 1.5  # neighbouring pairs overlap
    for u, v in ((a[1:], a[:-1]), (a[8:], a[:-8]), (a, b)):
        assert abs(float((u * v).sum()) - q * q * n) < pair


@pytest.mark.parametrize("ld", [65536, 65544, 65537])
def test_elements_past_32_bits(ld):
    T, d = 65600, 65536  # 4.3e9 elements
    x = torch.ones(T, ld, dtype=BF, device="cuda")[:, :d]
    y = moe.moe_dropout(x, 0.5, 1, 2)
    for row in (1, T // 2 + 1, T - 1):
        keep = keep_mask(512, 0.5, 1, 2, first=row * d)
        assert torch.equal((y[row, :512] != 0).cpu(), keep)


def test_in_place_streams_and_graph():
    g = torch.Generator().manual_seed(2)
    x, res = matrix(70, 520, BF, g), matrix(70, 520, BF, g)
    want = moe.moe_dropout(x, 0.2, 5, 6, residual=res)
    s = torch.cuda.Stream()
    x2, r2 = x.clone(), res.clone()
    s.wait_stream(torch.cuda.current_stream())
    moe.moe_dropout(x2, 0.2, 5, 6, residual=res, y=x2, stream=s)
    moe.moe_dropout(x, 0.2, 5, 6, residual=r2, y=r2, stream=s)
    s.synchronize()
    assert torch.equal(x2, want) and torch.equal(r2, want)
    # a captured call draws anew when the device counter is advanced
    ctr = torch.zeros(1, dtype=torch.int64, device="cuda")
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = moe.moe_dropout(x, 0.2, 5, 6, residual=res, offset_dev=ctr)
        ctr += 1
    for k in range(3):
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, moe.moe_dropout(x, 0.2, 5, 6 + k, residual=res))
