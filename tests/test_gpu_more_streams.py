"""The projections, the norms around a block and the calls that move rows: on a stream other than
the current one (what they allocate comes from that stream's memory), arguments that the Python
side refuses on the GPU, and two graphs that share a workspace."""
import pytest
import torch

from top_routing_grouped_02_gb300 import moe

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


def operands():
    torch.manual_seed(3)
    x, b, dy, du, gate = (torch.randn(100, 264, device="cuda").to(BF) for _ in range(5))
    w = torch.randn(264, device="cuda")
    W, bias = torch.randn(264, 520, device="cuda").mul_(0.06).to(BF), torch.randn(520, device="cuda")
    res = torch.randn(100, 520, device="cuda").to(BF)
    row = torch.randperm(300, device="cuda").int()
    return x, b, dy, du, gate, w, W, bias, res, row, torch.rand(100, 3, device="cuda")


def calls():
    x, b, dy, du, gate, w, W, bias, res, row, k = operands()
    _, _, rp, rq = moe.moe_block_norm(x, b, w, w, gate=gate, stats=True)
    xg = moe.moe_dispatch(x, row, 3)
    F = moe.moe_linear_train(x, W, bias, act="silu")[1]
    return {
        "norm": lambda s: moe.moe_block_norm(x, b, w, w, gate=gate, stats=True, stream=s),
        "norm_backward": lambda s: moe.moe_block_norm_backward(dy, du, x, b, w, w, rp, rq, gate=gate, stream=s),
        "dispatch": lambda s: (moe.moe_dispatch(x, row, 3, stream=s),),
        "dispatch_backward": lambda s: (moe.moe_dispatch_backward(xg, row, 3, residual=x, stream=s),),
        "combine": lambda s: (moe.moe_combine_weighted(xg, row, k, residual=x, stream=s),),
        "combine_backward": lambda s: moe.moe_combine_weighted_backward(dy, xg, row, k, stream=s),
        "linear": lambda s: (moe.moe_linear(x, W, bias, act="gelu", residual=res, stream=s),),
        "linear_few": lambda s: (moe.moe_linear(x[:3], W, bias, act="gelu", stream=s),),
        "linear_train": lambda s: (moe.moe_linear_train(x, W, bias, act="silu", residual=res, stream=s)[0],),
        "linear_backward": lambda s: moe.moe_linear_backward(res, x, W, F, bias_dtype=F32, stream=s),
    }


@pytest.mark.parametrize("name", ["norm", "norm_backward", "dispatch", "dispatch_backward", "combine", "combine_backward",
                                  "linear", "linear_few", "linear_train", "linear_backward"])
def test_memory_belongs_to_the_calls_stream(name):
    call = calls()[name]
    want = call(None)
    side = torch.cuda.Stream()
    big = torch.randn(4096, 4096, device="cuda")
    prod = torch.empty_like(big)
    call(side)
    sizes = (moe.lib().moe_block_norm_scratch_bytes(100, 264), moe.lib().moe_linear_workspace_bytes(100, 264, 520, 1))

    def scribble():
        junk = [torch.empty_like(t) for t in want for _ in range(4)]
        junk += [torch.empty(n // 4, device="cuda") for n in sizes for _ in range(3)]
        for j in junk:
            j.fill_(float("nan"))

    def busy():
        for _ in range(20):
            torch.mm(big, big, out=prod)

    torch.cuda.synchronize()
    # memory that the current stream has yet to write, given back on the host
    busy()
    scribble()
    got = call(side)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    # memory that the current stream asks for while the call waits on its own
    del got
    with torch.cuda.stream(side):
        busy()
    got = call(side)
    scribble()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_refusals():
    x, b, dy, du, gate, w, W, bias, res, row, k = operands()
    bad = [
        lambda: moe.moe_block_norm(x, b[:50], w, w), lambda: moe.moe_block_norm(x, b, w[:9], w), lambda: moe.moe_block_norm(x, b.half(), w, w),
        lambda: moe.moe_block_norm(x, b, gate=gate[:, :9]), lambda: moe.moe_block_norm(x, b, gate=gate[:, 0]),
        lambda: moe.moe_block_norm(x.t(), b.t()), lambda: moe.moe_block_norm(x, b, pre_norm=False, u=x),
        lambda: moe.moe_rmsnorm(x, y=b[:9]), lambda: moe.moe_block_norm(x.double(), b.double()),
        lambda: moe.moe_dispatch(x, row[:-1], 3), lambda: moe.moe_dispatch(x, row.long(), 3), lambda: moe.moe_dispatch(x, row, 0),
        lambda: moe.moe_dispatch(x, row, 3, xg=x.half()), lambda: moe.moe_dispatch(x, row, 3, xg=x[:, :9]),
        lambda: moe.moe_combine_weighted(x, row, k[:, :2]), lambda: moe.moe_combine_weighted(x, row, k.half()),
        lambda: moe.moe_combine_weighted(x, row, k, residual=x[:9]), lambda: moe.moe_combine_weighted(x, row, k, y=x[:9]),
        lambda: moe.moe_combine_weighted_backward(x, x, row, k, dz=x[:9]), lambda: moe.moe_combine_weighted_backward(x[:9], x, row, k),
        lambda: moe.moe_linear(x, W[:8]), lambda: moe.moe_linear(x, W.half()), lambda: moe.moe_linear(x, W, bias[:8]),
        lambda: moe.moe_linear(x, W, residual=res[:9]), lambda: moe.moe_linear(x, W, Y=res[:9]), lambda: moe.moe_linear(x, W, act="tanh"),
        lambda: moe.moe_linear(x[:, ::2], W[::2]), lambda: moe.moe_linear_backward(res, x, W, bias)]
    for i, call in enumerate(bad):
        with pytest.raises(ValueError):
            call()
            pytest.fail(f"call {i} was not refused")
    for call in (lambda: moe.moe_block_norm(x, b, w, w.to(BF)), lambda: moe.moe_block_norm(x, b, w.half()),
                 lambda: moe.moe_linear(x, W, bias.half()), lambda: moe.moe_linear(x.float(), W.float())):
        with pytest.raises(TypeError):
            call()
    for call in (lambda: moe.moe_dispatch(x, torch.zeros(900, dtype=torch.int32, device="cuda"), 9),
                 lambda: moe.moe_dispatch(x, row[:100], 1, xg=x), lambda: moe.moe_combine_weighted(x, row[:100], k[:, :1].contiguous(), y=x),
                 lambda: moe.moe_block_norm(x, b, y=x[:, :], u=x), lambda: moe.moe_linear(x[:, 4:].contiguous()[:, :256].contiguous()[1:], W[:256], Y=None, ws=x)):
        with pytest.raises(moe.MoeError):
            call()
    neither = torch.ones(2)  # no truth value
    for call in (lambda: moe.moe_block_norm(x, b, stats=neither), lambda: moe.moe_block_norm(x, b, post_norm=neither),
                 lambda: moe.moe_linear_backward(res, x, W, None, need_dx=neither)):
        with pytest.raises(RuntimeError, match="ambiguous"):
            call()


def test_two_graphs_share_a_workspace():
    """Replayed one after the other, in either order, each as a direct call."""
    x, _, _, _, _, _, W, bias, res, _, _ = operands()
    few = x[:3].contiguous()
    ws = moe.linear_workspace(100, 264, 520, train=True)
    V = W.t().contiguous()

    def first():
        y, F = moe.moe_linear_train(x, W, bias, act="gelu", residual=res, ws=ws)
        return y, *moe.moe_linear_backward(res, x, W, F, bias_dtype=F32, ws=ws)

    def second():
        return moe.moe_linear(few, W, bias, act="silu", ws=ws), moe.moe_linear(res, V, ws=ws)

    want = [first(), second()]
    graphs, outs = [], []
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        first(), second()
    torch.cuda.current_stream().wait_stream(side)
    for f in (first, second):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(f())
        graphs.append(g)
    for order in ((0, 1), (1, 0), (0, 0), (1, 1, 0)):
        for i in order:
            for t in outs[i]:
                t.fill_(float("nan"))
            graphs[i].replay()
            assert all(torch.equal(p, q) for p, q in zip(outs[i], want[i]))
    assert moe.moe_sync_check(ws) == (0, 0)
