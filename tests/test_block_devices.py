"""The sub-block calls take one device's tensors and streams: operands on another are refused
before the library sees a pointer. Tensors that only say where they would lie stand in for
those of a second GPU; no GPU is needed."""
import types

import pytest
import torch
from torch._subclasses.fake_tensor import FakeTensorMode

from top_routing_grouped_02_gb300 import _build, moe

BF = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def built():
    _build.build()


def on(device, *sizes, dtype=BF):
    with FakeTensorMode():
        return torch.empty(*sizes, dtype=dtype, device=device)


def operands(**where):
    """The calls' operands on cuda:0, but for those that `where` moves."""
    sizes = dict(x=(4, 64), y=(4, 64), dy=(4, 64), dres=(4, 64), gamma=(64,), beta=(64,), W1=(64, 128), W3=(64, 128),
                 W2=(128, 64), H=(4, 128))
    t = {k: on(where.get(k, "cuda:0"), *v) for k, v in sizes.items()}
    for k in ("mean", "rstd"):
        t[k] = on(where.get(k, "cuda:0"), 4, dtype=torch.float32)
    for k in ("F1", "F3"):
        t[k] = on(where.get(k, "cuda:0"), 4096, dtype=torch.float32)
    t["ctr"] = on(where.get("ctr", "cuda:0"), 1, dtype=torch.int64)
    for k in ("ws", "scratch"):
        t[k] = on(where.get(k, "cuda:0"), 1 << 20, dtype=torch.uint8)
    return types.SimpleNamespace(**t)


CALLS = {
    "layernorm": (lambda t, s: moe.moe_layernorm(t.x, t.gamma, t.beta, y=t.y, stream=s), ("x", "gamma", "beta", "y")),
    "layernorm_backward": (lambda t, s: moe.moe_layernorm_backward(t.dy, t.x, t.gamma, t.mean, t.rstd, dres=t.dres, dx=t.y,
                                                                   scratch=t.scratch, stream=s),
                           ("dy", "x", "gamma", "mean", "rstd", "dres", "y", "scratch")),
    "dropout": (lambda t, s: moe.moe_dropout(t.x, 0.1, 1, residual=t.dres, offset_dev=t.ctr, y=t.y, stream=s),
                ("x", "dres", "ctr", "y")),
    "dropout_backward": (lambda t, s: moe.moe_dropout_backward(t.dy, 0.1, 1, offset_dev=t.ctr, dx=t.y, stream=s),
                         ("dy", "ctr", "y")),
    "ffn": (lambda t, s: moe.moe_ffn(t.x, t.W1, t.W3, t.W2, ws=t.ws, Y=t.y, stream=s), ("x", "W1", "W3", "W2", "ws", "y")),
    "ffn_train": (lambda t, s: moe.moe_ffn_train(t.x, t.W1, t.W3, t.W2, ws=t.ws, stream=s), ("x", "W1", "W3", "W2", "ws")),
    "ffn_backward": (lambda t, s: moe.moe_ffn_backward(t.dy, t.x, t.W1, t.W3, t.W2, t.H, t.F1, t.F3, ws=t.ws, stream=s),
                     ("dy", "x", "W1", "W3", "W2", "H", "F1", "F3", "ws")),
}


@pytest.mark.parametrize("name", CALLS)
@pytest.mark.parametrize("other", ["cuda:1", "cpu"])
def test_operands_of_another_device(name, other):
    call, names = CALLS[name]
    for k in names:
        with pytest.raises(ValueError, match="device|CUDA tensor"):
            call(operands(**{k: other}), None)


@pytest.mark.parametrize("name", CALLS)
def test_stream_of_another_device(name):
    stream = types.SimpleNamespace(cuda_stream=0, device_index=1)
    with pytest.raises(ValueError, match="stream must belong"):
        CALLS[name][0](operands(), stream)


def test_workspace_and_stream_of_two_devices():
    stream = types.SimpleNamespace(cuda_stream=0, device_index=1, device=torch.device("cuda:1"))
    with pytest.raises(ValueError, match="stream must belong"):
        moe.ffn_workspace(4, 64, 128, device="cuda:0", stream=stream)
    with pytest.raises(ValueError, match="CUDA device"):
        moe.ffn_workspace(4, 64, 128, device="cpu")
