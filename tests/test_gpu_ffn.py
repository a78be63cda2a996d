"""The dense gated feed-forward block against its 64-bit form on a GB300."""
import pytest
import torch

from block_common import check_ffn, ffn
from top_routing_grouped_02_gb300 import moe

pytestmark = pytest.mark.gpu

BF, HF = torch.bfloat16, torch.float16
# (T, d, n): tokens on both sides of every padding of the weight-streaming kernel and
# of the switch to the tiled one, widths of one vector, ragged, and cut between SMs
SHAPES = [(1, 8, 8), (1, 256, 512), (2, 64, 136), (5, 1000, 72), (16, 136, 264), (17, 264, 1000),
          (32, 512, 2048), (33, 520, 1024), (64, 72, 520), (65, 128, 128), (100, 1000, 2728),
          (128, 2056, 136), (129, 64, 64), (200, 136, 72), (256, 256, 512), (300, 1000, 520),
          (513, 264, 136), (1030, 72, 328)]


def make(T, d, n, dt, seed=0):
    g = torch.Generator("cuda").manual_seed(T * 7 + d * 3 + n + seed)
    r = lambda *s, k=1.0: (torch.randn(*s, generator=g, device="cuda") * k).to(dt)  # noqa: E731
    return r(T, d), r(d, n, k=d ** -0.5), r(d, n, k=d ** -0.5), r(n, d, k=n ** -0.5), r(T, d)


def clean(ws):
    assert moe.moe_sync_check(ws) == (0, 0)


@pytest.mark.parametrize("dt", [BF, HF])
@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("T,d,n", SHAPES)
def test_forward(T, d, n, act, dt):
    x, W1, W3, W2, _ = make(T, d, n, dt)
    ws = moe.ffn_workspace(T, d, n)
    Y = moe.moe_ffn(x, W1, W3, W2, act, ws)
    clean(ws)
    check_ffn(Y, ffn(x, W1, W3, W2, act)["Y"], "Y")
    # the join counters are back at zero: the same workspace gives the same bits
    for _ in range(3):
        assert torch.equal(moe.moe_ffn(x, W1, W3, W2, act, ws), Y)


@pytest.mark.parametrize("dt", [BF, HF])
@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("T,d,n", SHAPES)
def test_training(T, d, n, act, dt):
    x, W1, W3, W2, dY = make(T, d, n, dt, 1)
    ws = moe.ffn_workspace(T, d, n, train=True)
    Y, H, A1, A3 = moe.moe_ffn_train(x, W1, W3, W2, act, ws)
    dX, dW1, dW3, dW2 = moe.moe_ffn_backward(dY, x, W1, W3, W2, H, A1, A3, act, ws=ws)
    clean(ws)
    ref = ffn(x, W1, W3, W2, act, dY)
    for name, got in (("Y", Y), ("dX", dX), ("dW1", dW1), ("dW3", dW3), ("dW2", dW2)):
        check_ffn(got, ref[name], name)
    # parts alone, and again: the same bits
    only = moe.moe_ffn_backward(dY, x, W1, W3, W2, H, A1, A3, act, need_dw=False, ws=ws)
    assert torch.equal(only[0], dX) and only[1] is None
    only = moe.moe_ffn_backward(dY, x, W1, W3, W2, H, A1, A3, act, need_dx=False, ws=ws)
    assert only[0] is None
    assert torch.equal(only[1], dW1) and torch.equal(only[2], dW3) and torch.equal(only[3], dW2)


@pytest.mark.parametrize("T,d,n", [(1, 4096, 14336), (48, 7168, 2048), (128, 1536, 4096), (512, 2048, 1408)])
def test_forward_at_working_sizes(T, d, n):
    x, W1, W3, W2, _ = make(T, d, n, BF, 2)
    ws = moe.ffn_workspace(T, d, n)
    Y = moe.moe_ffn(x, W1, W3, W2, "silu", ws)
    clean(ws)
    check_ffn(Y, ffn(x, W1, W3, W2, "silu")["Y"], "Y")


def test_one_workspace_for_several_shapes():
    shapes = [(128, 520, 1000), (1, 4096, 2048), (17, 64, 72), (300, 256, 512), (64, 2048, 264)]
    ws = max((moe.ffn_workspace(*s, train=True) for s in shapes), key=lambda w: w.numel())
    for _ in range(2):
        for s in shapes:
            x, W1, W3, W2, _ = make(*s, BF, 3)
            assert torch.equal(moe.moe_ffn(x, W1, W3, W2, "silu", ws), moe.moe_ffn(x, W1, W3, W2))
    clean(ws)


def test_empty():
    x, W1, W3, W2, dY = make(0, 64, 128, BF)
    ws = moe.ffn_workspace(0, 64, 128, train=True)
    assert moe.moe_ffn(x, W1, W3, W2, "silu", ws).shape == (0, 64)
    Y, H, A1, A3 = moe.moe_ffn_train(x, W1, W3, W2, "silu", ws)
    dX, dW1, dW3, dW2 = moe.moe_ffn_backward(dY, x, W1, W3, W2, H, A1, A3, "silu", ws=ws)
    assert dX.shape == (0, 64) and not dW1.any() and not dW3.any() and not dW2.any()


@pytest.mark.parametrize("T", [5, 64, 300])
def test_nonfinite_rows_stay_apart(T):
    x, W1, W3, W2, _ = make(T, 136, 264, BF, 4)
    want = moe.moe_ffn(x, W1, W3, W2)
    x = x.clone()
    x[1, 7] = float("nan")
    x[3, 130] = float("inf")
    y = moe.moe_ffn(x, W1, W3, W2)
    keep = [t for t in range(T) if t not in (1, 3)]
    assert torch.equal(y[keep], want[keep])
    assert torch.isnan(y[1]).all() and not torch.isfinite(y[3]).any()


@pytest.mark.parametrize("T", [3, 200])
def test_saturated_activations(T):
    # pre-activations of +-100: the sigmoid is 0 or 1 to the last bit, no overflow
    for act in ("silu", "gelu"):
        x = torch.ones(T, 64, device="cuda", dtype=BF)
        W1 = torch.full((64, 72), 100.0 / 64, device="cuda", dtype=BF)
        W1[:, 1::2] *= -1
        W3 = torch.full((64, 72), 1.0 / 64, device="cuda", dtype=BF)
        W2 = torch.full((72, 64), 1.0 / 64, device="cuda", dtype=BF)
        dY = torch.ones_like(x)
        ws = moe.ffn_workspace(T, 64, 72, train=True)
        Y, H, A1, A3 = moe.moe_ffn_train(x, W1, W3, W2, act, ws)
        grads = moe.moe_ffn_backward(dY, x, W1, W3, W2, H, A1, A3, act, ws=ws)
        ref = ffn(x, W1, W3, W2, act, dY)
        check_ffn(moe.moe_ffn(x, W1, W3, W2, act), ref["Y"], "Y")
        for name, got in zip(("Y", "dX", "dW1", "dW3", "dW2"), (Y,) + grads):
            want, slack = ref[name]
            assert torch.isfinite(got).all()
            assert ((got.double() - want).abs() <= 2.0 ** -8 * (want.abs() + slack) + slack + 1e-30).all(), name


def test_streams_and_graph():
    x, W1, W3, W2, dY = make(200, 264, 520, BF, 5)
    want = moe.moe_ffn_train(x, W1, W3, W2)
    wg = moe.moe_ffn_backward(dY, x, W1, W3, W2, *want[1:])
    xs = x[:7].contiguous()
    small = moe.moe_ffn(xs, W1, W3, W2)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    ws = [moe.ffn_workspace(200, 264, 520, train=True) for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(5):
        a = moe.moe_ffn(xs, W1, W3, W2, ws=ws[0])
        b = moe.moe_ffn(xs, W1, W3, W2, ws=ws[1], stream=side)
        torch.cuda.synchronize()
        assert torch.equal(a, small) and torch.equal(b, small)
    graph = torch.cuda.CUDAGraph()
    xin = torch.zeros_like(x)
    with torch.cuda.graph(graph):
        out = moe.moe_ffn_train(xin, W1, W3, W2, ws=ws[0])
        grads = moe.moe_ffn_backward(dY, xin, W1, W3, W2, *out[1:], ws=ws[0])
        s2 = moe.moe_ffn(xin[:7], W1, W3, W2, ws=ws[0])
    xin.copy_(x)
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    for p, q in zip(out + grads + (s2,), want + wg + (small,)):
        assert torch.equal(p, q)


def test_gradient_against_differences():
    # the loss <Y, dY> along random directions, by central differences in 64 bits; the
    # kernels' 16-bit roundings leave u times the gradient's norm
    T, d, n = 40, 72, 136
    x, W1, W3, W2, dY = make(T, d, n, BF, 6)
    out = moe.moe_ffn_train(x, W1, W3, W2, "gelu")
    grads = moe.moe_ffn_backward(dY, x, W1, W3, W2, *out[1:], "gelu")
    args = [t.double() for t in (x, W1, W3, W2)]
    g = torch.Generator("cuda").manual_seed(0)

    def loss(ts):
        a = ts[0] @ ts[1]
        return ((torch.nn.functional.gelu(a, approximate="tanh") * (ts[0] @ ts[2])) @ ts[3] * dY.double()).sum()

    h = 1e-5
    for k in range(4):
        u = torch.randn(args[k].shape, generator=g, device="cuda", dtype=torch.float64)
        plus, minus = ([t + s * h * u if j == k else t for j, t in enumerate(args)] for s in (1, -1))
        want = float(loss(plus) - loss(minus)) / (2 * h)
        got = grads[k].double()
        assert abs(float((got * u).sum()) - want) <= 4 * 1.5 * 2.0 ** -8 * float(got.norm())


def test_argument_checks():
    x, W1, W3, W2, _ = make(4, 64, 128, BF)
    for bad in ((x[:, :56], W1, W3, W2), (x, W1.half(), W3, W2), (x, W1, W3.t(), W2), (x, W1, W3, W1),
                (x.cpu(), W1, W3, W2)):
        with pytest.raises(ValueError):
            moe.moe_ffn(*bad)
    with pytest.raises(TypeError):
        moe.moe_ffn(x.float(), W1.float(), W3.float(), W2.float())
    with pytest.raises(ValueError):
        moe.moe_ffn(x, W1, W3, W2, "tanh")
    with pytest.raises(moe.MoeError):
        moe.moe_ffn(x, W1, W3, W2, ws=torch.zeros(1024, dtype=torch.uint8, device="cuda"))


def test_one_workspace_for_cut_tiles_of_many_shapes():
    # tiles that few pairs would take are cut; their join counters are back at zero after
    # each call, also where the rows of some warps lie outside
    ws = moe.ffn_workspace(2000, 1024, 4096, train=True)
    for T, d, n in [(1906, 184, 1824), (66, 216, 4096), (300, 1024, 512), (130, 1024, 1024), (66, 216, 4096),
                    (257, 520, 2056), (1906, 184, 1824)]:
        x, W1, W3, W2, dY = make(T, d, n, BF, T)
        want = None
        for w in (None, ws, ws):
            out = moe.moe_ffn_train(x, W1, W3, W2, "gelu", w)
            got = (out[0], out[1]) + moe.moe_ffn_backward(dY, x, W1, W3, W2, *out[1:], "gelu", ws=w)
            if want is None:
                want = got
            assert all(torch.equal(a, b) for a, b in zip(got, want)), (T, d, n)
    assert moe.moe_sync_check(ws)[0] == 0


@pytest.mark.parametrize("dt", [BF, HF])
@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("T,d,n", [(66, 4096, 256), (130, 4096, 200), (66, 216, 4096), (257, 136, 3000),
                                   (2700, 200, 136), (1906, 184, 1824)])
def test_tiles_of_many_segments(T, d, n, act, dt):
    # one or a few tiles and long reductions: five and more segments a tile, in each of the
    # products, with rows and columns past the tensors
    x, W1, W3, W2, dY = make(T, d, n, dt, 3)
    ws = moe.ffn_workspace(T, d, n, train=True)
    Y, H, F1, F3 = moe.moe_ffn_train(x, W1, W3, W2, act, ws)
    dX, dW1, dW3, dW2 = moe.moe_ffn_backward(dY, x, W1, W3, W2, H, F1, F3, act, ws=ws)
    clean(ws)
    ref = ffn(x, W1, W3, W2, act, dY)
    for name, got in (("Y", Y), ("dX", dX), ("dW1", dW1), ("dW3", dW3), ("dW2", dW2)):
        check_ffn(got, ref[name], name)
    for _ in range(3):  # the order of arrival does not matter
        again = moe.moe_ffn_backward(dY, x, W1, W3, W2, H, F1, F3, act, ws=ws)
        assert all(torch.equal(a, b) for a, b in zip(again, (dX, dW1, dW3, dW2)))
        assert torch.equal(moe.moe_ffn(x, W1, W3, W2, act, ws), Y)


@pytest.mark.parametrize("T", [48, 49, 64])
def test_forward_at_the_switch_of_large_weights(T):
    x, W1, W3, W2, _ = make(T, 4096, 11264, BF, 4)
    Y = moe.moe_ffn(x, W1, W3, W2)
    check_ffn(Y, ffn(x, W1, W3, W2, "silu")["Y"], "Y")


@pytest.mark.parametrize("T,d,n", [(3, 8200, 6088), (40, 8136, 6136)])
def test_few_tokens_with_ragged_large_weights(T, d, n):
    # long runs whose last tiles and units end past the weights
    x, W1, W3, W2, _ = make(T, d, n, BF, 5)
    ws = moe.ffn_workspace(T, d, n)
    Y = moe.moe_ffn(x, W1, W3, W2, "gelu", ws)
    clean(ws)
    check_ffn(Y, ffn(x, W1, W3, W2, "gelu")["Y"], "Y")
    assert torch.equal(moe.moe_ffn(x, W1, W3, W2, "gelu", ws), Y)
