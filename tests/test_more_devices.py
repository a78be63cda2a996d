"""The projections, the norms around a block and the calls that move rows take one device's
tensors and streams: operands on another are refused before the library sees a pointer (stand-ins
for a second GPU's tensors; no GPU is needed)."""
import types

import pytest
import torch
from torch._subclasses.fake_tensor import FakeTensorMode

from top_routing_grouped_02_gb300 import _build, moe

BF, F32, I32 = torch.bfloat16, torch.float32, torch.int32


@pytest.fixture(scope="module", autouse=True)
def built():
    _build.build()


def operands(**where):
    """The calls' operands on cuda:0, but for those that `where` moves."""
    shapes = dict(x=((4, 64), BF), y=((4, 64), BF), u=((4, 64), BF), b=((4, 64), BF), gate=((4, 64), BF), dy=((4, 64), BF),
                  du=((4, 64), BF), db=((4, 64), BF), post=((64,), F32), pre=((64,), F32), rp=((4,), F32), rq=((4,), F32),
                  z=((8, 64), BF), xg=((8, 64), BF), row=((8,), I32), w=((4, 2), F32), W=((64, 128), BF), bias=((128,), F32),
                  res=((4, 128), BF), Y=((4, 128), BF), F=((4096,), F32), ws=((1 << 20,), torch.uint8))
    with FakeTensorMode():
        return types.SimpleNamespace(**{k: torch.empty(s, dtype=d, device=where.get(k, "cuda:0")) for k, (s, d) in shapes.items()})


CALLS = {
    "block_norm": (lambda t, s: moe.moe_block_norm(t.x, t.b, t.post, t.pre, gate=t.gate, y=t.y, u=t.u, stream=s),
                   ("x", "b", "post", "pre", "gate", "y", "u")),
    "block_norm_backward": (lambda t, s: moe.moe_block_norm_backward(t.dy, t.du, t.x, t.b, t.post, t.pre, t.rp, t.rq, gate=t.gate,
                                                                     dx=t.y, db=t.db, scratch=t.ws, stream=s),
                            ("dy", "du", "x", "b", "post", "pre", "rp", "rq", "gate", "y", "db", "ws")),
    "rmsnorm": (lambda t, s: moe.moe_rmsnorm(t.x, t.pre, y=t.y, stream=s), ("x", "pre", "y")),
    "rmsnorm_backward": (lambda t, s: moe.moe_rmsnorm_backward(t.du, t.x, t.pre, t.rq, dres=t.dy, dx=t.y, scratch=t.ws, stream=s),
                         ("du", "x", "pre", "rq", "dy", "y", "ws")),
    "dispatch": (lambda t, s: moe.moe_dispatch(t.x, t.row, 2, xg=t.xg, stream=s), ("x", "row", "xg")),
    "dispatch_backward": (lambda t, s: moe.moe_dispatch_backward(t.z, t.row, 2, residual=t.x, dx=t.y, stream=s), ("z", "row", "x", "y")),
    "combine": (lambda t, s: moe.moe_combine_weighted(t.z, t.row, t.w, residual=t.x, y=t.y, stream=s), ("z", "row", "w", "x", "y")),
    "combine_backward": (lambda t, s: moe.moe_combine_weighted_backward(t.dy, t.z, t.row, t.w, dz=t.xg, stream=s),
                         ("dy", "z", "row", "w", "xg")),
    "linear": (lambda t, s: moe.moe_linear(t.x, t.W, t.bias, residual=t.res, ws=t.ws, Y=t.Y, stream=s),
               ("x", "W", "bias", "res", "ws", "Y")),
    "linear_train": (lambda t, s: moe.moe_linear_train(t.x, t.W, t.bias, act="silu", residual=t.res, ws=t.ws, stream=s),
                     ("x", "W", "bias", "res", "ws")),
    "linear_backward": (lambda t, s: moe.moe_linear_backward(t.Y, t.x, t.W, t.F, ws=t.ws, stream=s), ("Y", "x", "W", "F", "ws")),
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
        moe.linear_workspace(4, 64, 128, device="cuda:0", stream=stream)
    with pytest.raises(ValueError, match="CUDA device"):
        moe.linear_workspace(4, 64, 128, device="cpu")
