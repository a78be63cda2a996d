"""Rows to expert order and back with weights, and the gradients, against 64-bit plain forms."""
import pytest
import torch

import rows_common as plain
from block_common import assert_close, matrix
from top_routing_grouped_02_gb300 import moe

pytestmark = pytest.mark.gpu

BF, FP16, F32 = torch.bfloat16, torch.float16, torch.float32

# T, K, E, d, type, row stride, share of slots without a row
CASES = [
    (1, 1, 1, 8, BF, None, 0.0), (1, 2, 8, 4096, BF, None, 0.0), (1, 8, 64, 7168, FP16, None, 0.25),
    (5, 3, 7, 1, BF, None, 0.2), (5, 3, 7, 7, FP16, None, 0.2), (3, 8, 9, 9, F32, None, 0.0),
    (33, 2, 5, 255, BF, 257, 0.1), (33, 4, 9, 256, BF, 264, 0.5), (17, 5, 11, 1023, F32, 1026, 0.1),
    (64, 6, 16, 1000, FP16, 1002, 0.0), (300, 7, 20, 130, BF, 132, 0.3), (257, 8, 32, 1536, BF, None, 0.0),
    (40, 4, 40, 96, F32, None, 1.0), (9, 2, 4, 2050, F32, None, 0.0), (2000, 1, 3, 72, BF, None, 0.4),
    (130, 3, 8, 513, FP16, 513, 0.1),
]
IDS = [f"T{c[0]}K{c[1]}d{c[3]}ld{c[5] or c[3]}-{str(c[4])[6:]}-{c[6]}" for c in CASES]


def inputs(case):
    T, K, E, d, dt, ld, drop = case
    gen = torch.Generator().manual_seed(T * 1000 + d)
    row, used = plain.slot_map(T, K, E, drop, gen)
    w = torch.randn(T, K, generator=gen)
    w[(row < 0).view(T, K)] = float("nan")  # not read into anything
    mats = {k: matrix(n, d, dt, gen, ld) for k, n in
            (("x", T), ("z", T * K), ("res", T), ("dy", T), ("xg", T * K), ("dz", T * K))}
    mats["z"][used:] = float("nan")  # rows that no slot names
    return row, used, w, mats


@pytest.mark.parametrize("case", CASES, ids=IDS)
def test_dispatch(case):
    T, K, _, d, dt, ld, drop = case
    row, used, _, m = inputs(case)
    want = plain.dispatch(m["x"].cpu(), row, K, m["xg"].cpu())
    if drop == 0:
        got = moe.moe_dispatch(m["x"], row.cuda(), K)
        assert got.shape == (T * K, d) and torch.equal(got.double().cpu(), want)
    got = moe.moe_dispatch(m["x"], row.cuda(), K, xg=m["xg"])
    assert got.data_ptr() == m["xg"].data_ptr() and torch.equal(got.double().cpu(), want)


@pytest.mark.parametrize("case", CASES, ids=IDS)
def test_dispatch_backward(case):
    T, K, _, d, dt, ld, _ = case
    row, _, _, m = inputs(case)
    for res in (None, m["res"]):
        y = moe.moe_dispatch_backward(m["z"], row.cuda(), K, residual=res)
        want, size = plain.combine(m["z"].cpu(), row, K, None if res is None else res.cpu())
        assert_close(y, want, size, K, "dx")


@pytest.mark.parametrize("case", CASES, ids=IDS)
def test_combine(case):
    T, K, _, d, dt, ld, _ = case
    row, _, w, m = inputs(case)
    for res in (None, m["res"]):
        y = moe.moe_combine_weighted(m["z"], row.cuda(), w.cuda(), residual=res)
        want, size = plain.combine(m["z"].cpu(), row, w, None if res is None else res.cpu())
        # K fused multiply-adds and the residual's sum
        assert_close(y, want, size, K + 1, "y")
    want = y.clone()
    y = moe.moe_combine_weighted(m["z"], row.cuda(), w.cuda(), residual=m["res"], y=m["res"])
    assert y.data_ptr() == m["res"].data_ptr() and torch.equal(y, want)


@pytest.mark.parametrize("case", CASES, ids=IDS)
def test_combine_backward(case):
    T, K, _, d, dt, ld, drop = case
    row, used, w, m = inputs(case)
    want_dz, want_dw, size = plain.combine_backward(m["dy"].cpu(), m["z"].cpu(), row, w, m["dz"].cpu())
    dz, dw = moe.moe_combine_weighted_backward(m["dy"], m["z"], row.cuda(), w.cuda(), dz=m["dz"])
    assert dz.data_ptr() == m["dz"].data_ptr()
    # one product in fp32, then rounded
    assert_close(dz[:used], want_dz[:used], want_dz[:used].abs(), 1, "dz")
    assert torch.equal(dz[used:].double().cpu(), want_dz[used:])
    # a chain of at most d / 32 + 8 products a lane, five sums over lanes and seven over warps
    assert_close(dw, want_dw, size, d / 32 + 20, "dw")
    assert not dw.cpu()[(row < 0).view(T, K)].any()
    kept = dz.clone()
    dz, _ = moe.moe_combine_weighted_backward(m["dy"], m["z"], row.cuda(), w.cuda(), dz=m["z"])
    assert torch.equal(dz[:used], kept[:used])


def test_gradients_by_differences():
    """The combine's and the dispatch's gradients against differences of the calls themselves."""
    T, K, d = 6, 3, 40
    gen = torch.Generator().manual_seed(3)
    row, _ = plain.slot_map(T, K, 5, 0.1, gen)
    row = row.cuda()
    w, z, dy = (torch.randn(*s, generator=gen).cuda() for s in ((T, K), (T * K, d), (T, d)))
    dz0 = torch.zeros_like(z)
    dz, dw = moe.moe_combine_weighted_backward(dy, z, row, w, dz=dz0)

    def loss(z, w):
        return float((moe.moe_combine_weighted(z, row, w).double() * dy.double()).sum())

    for name, value, grad in (("z", z, dz), ("w", w, dw)):
        step = torch.randn(value.shape, generator=gen).cuda()
        h = 2.0 ** -6  # the loss is linear in each: only roundings of about 2^-24 of its terms remain
        plus, minus = (loss(*((value + s * step, w) if name == "z" else (z, value + s * step))) for s in (h, -h))
        want = float((grad.double() * step.double()).sum())
        terms = float((grad.double() * step.double()).abs().sum()) + abs(plus) + abs(minus) + T * d
        assert abs((plus - minus) / (2 * h) - want) <= 2 ** -20 / h * terms, name


def test_map_values_outside_the_rows():
    x = torch.arange(8.0, device="cuda").view(2, 4)
    row = torch.tensor([1, -1, 2, 2 ** 31 - 1], dtype=torch.int32, device="cuda")
    xg = torch.full((2, 4), 7.0, device="cuda")
    moe.moe_dispatch(x, row, 2, xg=xg)
    assert xg.tolist() == [[7.0] * 4, [0.0, 1.0, 2.0, 3.0]]
    y = moe.moe_combine_weighted(xg, row, torch.full((2, 2), 2.0, device="cuda"))
    assert y.tolist() == [[0.0, 2.0, 4.0, 6.0], [0.0] * 4]
    none = torch.empty(0, 4, device="cuda")
    assert moe.moe_dispatch_backward(none, row, 2, residual=x).tolist() == x.tolist()
    moe.moe_dispatch(x, row, 2, xg=none)


def test_no_tokens():
    row = torch.empty(0, dtype=torch.int32, device="cuda")
    x = torch.empty(0, 16, device="cuda", dtype=BF)
    assert moe.moe_dispatch(x, row, 2).shape == (0, 16)
    w = torch.empty(0, 2, device="cuda")
    assert moe.moe_combine_weighted(x, row, w).shape == (0, 16)
    dz, dw = moe.moe_combine_weighted_backward(x, x, row, w)
    assert dz.shape == (0, 16) and dw.shape == (0, 2)


def test_maps_of_the_grouping():
    """moe_route and moe_permute's maps: the rows of an expert are its tokens', ascending."""
    T, d, E, K = 100, 64, 8, 2
    g = torch.Generator("cuda").manual_seed(1)
    x = torch.randn(T, d, generator=g, device="cuda").bfloat16()
    Wr = torch.randn(d, E, generator=g, device="cuda")
    idx, w, _ = moe.moe_route(x, Wr, K)
    p = moe.moe_permute(idx, E)
    xg = moe.moe_dispatch(x, p["row_of_slot"], K)
    assert torch.equal(xg, x[p["perm_token"].long()])
    y = moe.moe_combine_weighted(xg, p["row_of_slot"], w)
    want, size = plain.combine(xg.cpu(), p["row_of_slot"].cpu(), w.cpu())
    assert_close(y, want, size, K + 1, "y")


def test_offsets_past_32_bits():
    """Rows more than 2^31 elements into their matrices (9 GB of fp16 behind a view)."""
    d, ld, rows = 24, 1 << 26, 66
    big = torch.empty(rows * ld, dtype=FP16, device="cuda").view(rows, ld)[:, :d]
    x = torch.randn(33, d, device="cuda").half()
    row = torch.arange(rows, dtype=torch.int32).flip(0).cuda()
    moe.moe_dispatch(x, row, 2, xg=big)
    assert torch.equal(big.flip(0).reshape(33, 2, d), x[:, None].expand(33, 2, d))
    w = torch.rand(33, 2, device="cuda")
    y = moe.moe_combine_weighted(big, row, w)
    want, size = plain.combine(big.cpu(), row.cpu(), w.cpu())
    assert_close(y, want, size, 3, "y")


def test_captured_calls_and_streams():
    """Captured and replayed on new values; and a call on a given stream."""
    T, K, d = 50, 3, 104
    gen = torch.Generator().manual_seed(9)
    row, _ = plain.slot_map(T, K, 9, 0.0, gen)
    row, x = row.cuda(), torch.randn(T, d, generator=gen).cuda().bfloat16()
    w = torch.rand(T, K, generator=gen).cuda()

    def step():
        xg = moe.moe_dispatch(x, row, K)
        y = moe.moe_combine_weighted(xg, row, w, residual=x)
        return y, *moe.moe_combine_weighted_backward(y, xg, row, w)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for seed in (1, 2):
        x.copy_(torch.randn(T, d, generator=gen).bfloat16())
        graph.replay()
        for a, b in zip(out, step()):
            assert torch.equal(a, b)
    want = moe.moe_combine_weighted(out[2 - 1], row, w)
    side.wait_stream(torch.cuda.current_stream())
    got = moe.moe_combine_weighted(out[1], row, w, stream=side)
    side.synchronize()
    assert torch.equal(got, want)
