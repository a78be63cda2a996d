"""Calls of the sub-block on a stream other than the current one: what they allocate
(outputs, scratch, a workspace made for the call) comes from that stream's memory."""
import pytest
import torch

from top_routing_grouped_02_gb300 import moe

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


def calls():
    torch.manual_seed(3)
    x = torch.randn(100, 264, device="cuda").to(BF)
    dy = torch.randn(100, 264, device="cuda").to(BF)
    w = torch.randn(264, device="cuda")
    W1, W3 = (torch.randn(264, 520, device="cuda").mul_(0.06).to(BF) for _ in range(2))
    W2 = torch.randn(520, 264, device="cuda").mul_(0.04).to(BF)
    _, mean, rstd = moe.moe_layernorm(x, w, w, stats=True)
    saved = moe.moe_ffn_train(x, W1, W3, W2)[1:]
    return {
        "norm": lambda s: moe.moe_layernorm(x, w, w, stats=True, stream=s),
        "norm_backward": lambda s: moe.moe_layernorm_backward(dy, x, w, mean, rstd, dres=dy, stream=s),
        "dropout": lambda s: (moe.moe_dropout(x, 0.3, 1, 2, residual=dy, stream=s),),
        "dropout_backward": lambda s: (moe.moe_dropout_backward(x, 0.3, 1, 2, stream=s),),
        "ffn": lambda s: (moe.moe_ffn(x, W1, W3, W2, stream=s),),
        "ffn_few": lambda s: (moe.moe_ffn(x[:5], W1, W3, W2, stream=s),),
        "ffn_train": lambda s: moe.moe_ffn_train(x, W1, W3, W2, stream=s),
        "ffn_backward": lambda s: moe.moe_ffn_backward(dy, x, W1, W3, W2, *saved, stream=s),
    }


@pytest.mark.parametrize("name", ["norm", "norm_backward", "dropout", "dropout_backward", "ffn", "ffn_few",
                                  "ffn_train", "ffn_backward"])
def test_memory_belongs_to_the_calls_stream(name):
    call = calls()[name]
    want = call(None)
    side = torch.cuda.Stream()
    big = torch.randn(4096, 4096, device="cuda")
    prod = torch.empty_like(big)
    call(side)
    scratch = moe.lib().moe_layernorm_scratch_bytes(100, 264)
    workspace = moe.lib().moe_ffn_workspace_bytes(100, 264, 520, 1)

    def scribble():
        junk = [torch.empty_like(t) for t in want for _ in range(4)]
        junk += [torch.empty(n // 4, device="cuda") for n in (scratch, workspace) for _ in range(3)]
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
