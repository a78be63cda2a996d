"""Projections with bias, activation and residual, and their gradients, against 64 bits."""
import pytest
import torch

from block_common import HALF, TINY, matrix
from linear_common import linear
from top_routing_grouped_02_gb300 import moe

pytestmark = pytest.mark.gpu

BF, FP16, F32 = torch.bfloat16, torch.float16, torch.float32

# T, k, n, type, bias type (None: no bias), activation, residual
CASES = [
    (1, 8, 8, BF, BF, None, True), (1, 128, 4096, BF, F32, "silu", True), (1, 4096, 136, FP16, FP16, "gelu", False),
    (2, 64, 128, BF, None, None, False), (16, 1000, 2728, FP16, F32, "gelu", True), (17, 72, 40, BF, BF, "silu", True),
    (33, 2048, 1032, BF, F32, None, True), (48, 520, 264, FP16, None, "silu", False), (49, 520, 264, FP16, FP16, "gelu", True),
    (64, 7168, 256, BF, BF, "gelu", True), (100, 8, 8, BF, F32, "silu", True), (130, 4096, 128, BF, BF, None, True),
    (255, 640, 768, FP16, F32, "gelu", False), (256, 256, 256, BF, None, "silu", True), (257, 136, 520, BF, F32, "gelu", True),
    (777, 1000, 2728, BF, F32, "gelu", True), (1030, 2048, 200, FP16, FP16, "silu", True), (2100, 136, 8, BF, BF, None, True),
    (520, 8, 1500 * 8, BF, F32, "silu", False),
    # dX and dW in one launch and in two; tails in every dimension
    (300, 520, 264, BF, BF, "silu", True), (520, 264, 2056, FP16, FP16, None, False), (65, 2568, 1032, BF, F32, "gelu", True),
    (1, 264, 520, BF, BF, "gelu", False),
]
IDS = ["x".join(map(str, c[:3])) + f"-{str(c[3])[6:]}-{str(c[4])[6:] if c[4] else 'nobias'}-{c[5]}{'-res' if c[6] else ''}"
       for c in CASES]


def inputs(case):
    T, k, n, dt, bt, _, res = case
    gen = torch.Generator().manual_seed(T * 7 + k * 13 + n)
    return dict(x=matrix(T, k, dt, gen), W=matrix(k, n, dt, gen, scale=k ** -0.5),
                bias=None if bt is None else matrix(1, n, bt, gen, scale=0.5)[0].contiguous(),
                res=matrix(T, n, dt, gen, scale=2.0) if res else None, dY=matrix(T, n, dt, gen))


def check(got, ref, name):
    """Every element within its bound."""
    want, slack = (v.cuda() for v in ref)
    g = got.double()
    assert torch.isfinite(g).all(), f"{name}: not finite"
    bound = HALF[got.dtype] * (want.abs() + slack) + slack + TINY[got.dtype]
    err = (g - want).abs()
    assert (err <= bound).all(), f"{name}: {int((err > bound).sum())} off, worst {float((err / bound).max()):.3f} of its bound"


def unblocked(f, T, n):
    """[T, n] from blocks of 32 x 32: block, 8 fours of columns, 32 rows, 4 columns."""
    nb = (n + 31) // 32
    return f.view((T + 31) // 32, nb, 8, 32, 4).permute(0, 3, 1, 2, 4).reshape(-1, nb * 32)[:T, :n]


def reference(m, act):
    return linear(m["x"].cpu(), m["W"].cpu(), None if m["bias"] is None else m["bias"].cpu(), act,
                  None if m["res"] is None else m["res"].cpu(), m["dY"].cpu())


@pytest.mark.parametrize("case", CASES, ids=IDS)
def test_forward_and_backward(case):
    T, k, n, dt, bt, act, _ = case
    m = inputs(case)
    ref = reference(m, act)
    ws = moe.linear_workspace(T, k, n, train=True)
    y = moe.moe_linear(m["x"], m["W"], m["bias"], act=act, residual=m["res"])
    check(y, ref["Y"], "Y")
    y, f = moe.moe_linear_train(m["x"], m["W"], m["bias"], act=act, residual=m["res"], ws=ws)
    check(y, ref["Y"], "Y of training")
    assert (f is None) == (act is None)
    if f is not None:
        check(unblocked(f, T, n), ref["F"], "F")
    dX, dW, db = moe.moe_linear_backward(m["dY"], m["x"], m["W"], f, bias_dtype=bt, ws=ws)
    check(dX, ref["dX"], "dX")
    check(dW, ref["dW"], "dW")
    assert (db is None) == (bt is None)
    if db is not None:
        check(db, ref["dbias"], "dbias")
    assert moe.moe_sync_check(ws) == (0, 0)
    # the same again, and parts of it: the workspace is as it was
    again = moe.moe_linear_backward(m["dY"], m["x"], m["W"], f, bias_dtype=bt, ws=ws)
    assert all(p is q is None or torch.equal(p, q) for p, q in zip((dX, dW, db), again))
    one = moe.moe_linear_backward(m["dY"], m["x"], m["W"], f, need_dw=False, ws=ws)
    check(one[0], ref["dX"], "dX alone")  # (its sums may be in another order beside dW)
    assert one[1] is None and one[2] is None
    if bt is not None:  # the bias' gradient alone takes a kernel of its own
        check(moe.moe_linear_backward(m["dY"], m["x"], m["W"], f, bias_dtype=bt, need_dx=False, need_dw=False, ws=ws)[2],
              ref["dbias"], "dbias alone")
    one = moe.moe_linear_backward(m["dY"], m["x"], m["W"], f, need_dx=False, ws=ws)
    assert one[0] is None
    check(one[1], ref["dW"], "dW alone")
    # onto the residual, with a workspace of more tokens
    if m["res"] is not None:
        want = moe.moe_linear(m["x"], m["W"], m["bias"], act=act, residual=m["res"], ws=ws)
        got = moe.moe_linear(m["x"], m["W"], m["bias"], act=act, residual=m["res"], Y=m["res"], ws=ws)
        assert got.data_ptr() == m["res"].data_ptr() and torch.equal(got, want)


@pytest.mark.parametrize("act", [None, "silu", "gelu"])
def test_gradients_by_differences(act):
    """dX, dW and dbias against differences of the 64-bit formula at the kernels' inputs."""
    T, k, n = 70, 64, 72
    m = inputs((T, k, n, FP16, F32, act, False))
    ref = reference(m, act)
    y, f = moe.moe_linear_train(m["x"], m["W"], m["bias"], act=act)
    dX, dW, db = moe.moe_linear_backward(m["dY"], m["x"], m["W"], f, bias_dtype=F32)
    x, W, b, dY = (m[v].double().cpu() for v in ("x", "W", "bias", "dY"))

    def loss(x, W, b):
        from linear_common import act as formula
        return float((formula(x @ W + b, act)[0] * dY).sum())

    gen = torch.Generator().manual_seed(1)
    for i, (name, grad) in enumerate((("dX", dX), ("dW", dW), ("dbias", db))):
        step = torch.randn(grad.shape, generator=gen).double()
        h = 1e-5
        args = [[v + s * h * step if j == i else v for j, v in enumerate((x, W, b))] for s in (1, -1)]
        want = (loss(*args[0]) - loss(*args[1])) / (2 * h)
        value, slack = ref[name]
        bound = (slack + HALF[grad.dtype] * (value.abs() + slack)) * step.abs()
        # the difference itself: h^2 of a third derivative, and 2^-52 of the loss over h
        assert abs(float((grad.double().cpu() * step).sum()) - want) <= float(bound.sum()) + 1e-4, name


def test_infinities_and_empty():
    """A residual's infinities and NaN stay in their elements; no tokens."""
    m = inputs((50, 128, 64, BF, BF, "gelu", True))
    clean = moe.moe_linear(m["x"], m["W"], m["bias"], act="gelu", residual=m["res"])
    m["res"][3, 5], m["res"][49, 63] = float("inf"), float("nan")
    y = moe.moe_linear(m["x"], m["W"], m["bias"], act="gelu", residual=m["res"])
    bad = ~torch.isfinite(y)
    assert bad.nonzero().tolist() == [[3, 5], [49, 63]] and torch.equal(y[~bad], clean[~bad])
    for T in (1, 50):  # a very negative pre-activation: 0, and its derivative too
        b = torch.full((64,), -3e4, device="cuda")
        for act in ("silu", "gelu"):
            y, f = moe.moe_linear_train(m["x"][:T], m["W"], b, act=act)
            assert not y.any() and not unblocked(f, T, 64).any()
            assert not moe.moe_linear(m["x"][:T], m["W"], b, act=act).any()
            y, f = moe.moe_linear_train(m["x"][:T], m["W"], -b, act=act)
            assert (unblocked(f, T, 64) == 1).all() and torch.isfinite(y).all()
    none = torch.empty(0, 128, dtype=BF, device="cuda")
    y, f = moe.moe_linear_train(none, m["W"], m["bias"], act="silu")
    assert y.shape == (0, 64) and f.shape == (0,)
    dX, dW, db = moe.moe_linear_backward(y, none, m["W"], f, bias_dtype=F32)
    assert dX.shape == (0, 128) and dW.shape == (128, 64) and not dW.any() and not db.any()


def test_workspace_serves_fewer_tokens_and_other_calls():
    k, n = 512, 1032
    ws = moe.linear_workspace(600, k, n, train=True)
    for T in (600, 1, 48, 49, 64, 300):
        m = inputs((T, k, n, BF, F32, "silu", True))
        check(moe.moe_linear(m["x"], m["W"], m["bias"], act="silu", residual=m["res"], ws=ws), reference(m, "silu")["Y"], f"T={T}")
    small = moe.linear_workspace(16, k, n)
    with pytest.raises(moe.MoeError):
        moe.moe_linear(m["x"], m["W"], ws=small)
    assert moe.moe_sync_check(ws) == (0, 0)


def test_leading_dimensions():
    gen = torch.Generator().manual_seed(2)
    x = matrix(6, 64, BF, gen).view(2, 3, 64)
    W, b = matrix(64, 72, BF, gen), matrix(1, 72, BF, gen)[0].contiguous()
    y, f = moe.moe_linear_train(x, W, b, act="gelu")
    assert y.shape == (2, 3, 72)
    assert torch.equal(moe.moe_linear(x, W, b, act="gelu"), moe.moe_linear(x.view(6, 64), W, b, act="gelu").view(2, 3, 72))
    dX, dW, db = moe.moe_linear_backward(y, x, W, f, bias_dtype=BF)
    assert dX.shape == x.shape and dW.shape == W.shape and db.dtype == BF


@pytest.mark.parametrize("T", [4, 200])
def test_captured_calls_and_streams(T):
    k, n = 1024, 1032
    m = inputs((T, k, n, BF, F32, "silu", True))
    ws = moe.linear_workspace(T, k, n, train=True)
    gen = torch.Generator().manual_seed(5)

    def step():
        y = moe.moe_linear(m["x"], m["W"], m["bias"], act="silu", residual=m["res"], ws=ws)
        y2, f = moe.moe_linear_train(m["x"], m["W"], m["bias"], act="silu", residual=m["res"], ws=ws)
        return y, y2, *moe.moe_linear_backward(m["dY"], m["x"], m["W"], f, bias_dtype=F32, ws=ws)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for _ in range(2):
        m["x"].copy_(matrix(T, k, BF, gen))
        graph.replay()
        for p, q in zip(out, step()):
            assert torch.equal(p, q)
    want = moe.moe_linear(m["x"], m["W"], ws=ws)
    side.wait_stream(torch.cuda.current_stream())
    got = moe.moe_linear(m["x"], m["W"], stream=side)
    side.synchronize()
    assert torch.equal(got, want)
