"""Refusals of the projections, and the plain gradients of their tests (no GPU needed)."""
import pytest
import torch

from linear_common import act as formula
from linear_common import linear
from top_routing_grouped_02_gb300 import _build, moe

INVALID, SHAPE, SMALL = 1, 2, 3
A = [(i + 1) << 24 for i in range(12)]  # aligned addresses that are never read
BIG = 1 << 40


@pytest.fixture(scope="module")
def lib():
    # the addresses are made up: a call that passed its checks would use them on a GPU
    if torch.cuda.is_available():
        pytest.skip("refusals are tested where there is no GPU")
    _build.build()
    return moe.lib()


def fwd(lib, X=A[0], W=A[1], b=A[2], r=A[3], T=4, k=64, n=128, act=0, t=0, bt=0, Y=A[4], ws=A[6], nbytes=BIG):
    return lib.moe_linear_forward(X, W, b, r, T, k, n, act, t, bt, Y, ws, nbytes, None)


def train(lib, X=A[0], W=A[1], b=A[2], r=A[3], T=4, k=64, n=128, act=0, t=0, bt=0, Y=A[4], F=A[5], ws=A[6], nbytes=BIG):
    return lib.moe_linear_forward_train(X, W, b, r, T, k, n, act, t, bt, Y, F, ws, nbytes, None)


def bwd(lib, dY=A[3], X=A[0], W=A[1], F=A[5], T=4, k=64, n=128, t=0, bt=0, dX=A[7], dW=A[8], db=A[9], ws=A[6], nbytes=BIG):
    return lib.moe_linear_backward(dY, X, W, F, T, k, n, t, bt, dX, dW, db, ws, nbytes, None)


COMMON = [dict(X=None), dict(W=None), dict(X=A[0] + 8), dict(W=A[1] + 8), dict(T=-1), dict(k=0), dict(n=0), dict(t=3),
          dict(bt=1), dict(t=1, bt=0), dict(ws=None), dict(ws=A[6] + 128)]
SHAPES = [dict(k=60), dict(n=132), dict(k=(1 << 20) + 8), dict(n=(1 << 20) + 8), dict(t=2, bt=2), dict(T=(1 << 30) + 1)]


def test_refusals(lib):
    for call in (fwd, train, bwd):
        ok = call(lib)
        assert ok not in (INVALID, SHAPE, SMALL)
        for bad in COMMON:
            assert call(lib, **bad) == INVALID, (call, bad)
        for bad in SHAPES:
            assert call(lib, **bad) == SHAPE, (call, bad)
        assert call(lib, nbytes=1 << 10) == SMALL
        assert call(lib, bt=2) == ok
    ok = fwd(lib)
    for call in (fwd, train):
        for bad in (dict(Y=None), dict(Y=A[4] + 8), dict(b=A[2] + 8), dict(r=A[3] + 8), dict(act=3), dict(act=-1), dict(Y=A[0])):
            assert call(lib, **bad) == INVALID, (call, bad)
        assert call(lib, b=None, r=None) == ok and call(lib, Y=A[3]) == ok
        assert call(lib, T=0, X=None, Y=None, ws=None) == 0
    assert fwd(lib, act=2) == ok and train(lib, act=2, F=None) == ok
    for bad in (dict(act=2), dict(F=None), dict(F=A[5] + 8), dict(F=A[4])):
        assert train(lib, **bad) == INVALID, bad
    for bad in (dict(dY=None), dict(dY=A[3] + 8), dict(F=A[5] + 8), dict(dX=A[7] + 8), dict(dW=A[8] + 8), dict(db=A[9] + 1),
                dict(bt=2, db=A[9] + 2), dict(dX=A[0]), dict(dX=A[3]), dict(dW=A[1]), dict(dX=A[5])):
        assert bwd(lib, **bad) == INVALID, bad
    for good in (dict(F=None), dict(dX=None, W=None), dict(dW=None, X=None), dict(db=None)):
        assert bwd(lib, **good) == ok, good


def test_workspace_sizes(lib):
    size = lib.moe_linear_workspace_bytes
    assert size(4, 60, 64, 0) == 0 and size(-1, 64, 64, 0) == 0 and size(4, 64, 64, 3) == size(4, 64, 64, 1)
    for k, n in ((8, 8), (64, 4096), (14336, 4096), (1 << 20, 8), (8, 1 << 20)):
        for train_ in (0, 1):
            last = 0
            for T in (0, 1, 16, 17, 48, 49, 64, 65, 1000, 100000):
                assert size(T, k, n, train_) >= last, (T, k, n)  # serves fewer tokens
                last = size(T, k, n, train_)
            assert size(64, k, n, 1) >= size(64, k, n, 0)
    # a layer of ordinary size: the parts of cut tiles, no product of T, k and n
    assert size(4096, 4096, 14336, 0) < 64 << 20


@pytest.mark.parametrize("name", [None, "silu", "gelu"])
def test_plain_gradients(name):
    gen = torch.Generator().manual_seed(3)
    T, k, n = 5, 8, 16
    x, W, dY = (torch.randn(*s, generator=gen).double() for s in ((T, k), (k, n), (T, n)))
    b = torch.randn(n, generator=gen).double()
    x, W, dY = (v.bfloat16() for v in (x, W, dY))
    leaves = [v.double().requires_grad_() for v in (x, W, b)]
    y, df = formula(leaves[0] @ leaves[1] + leaves[2], name)
    y.backward(dY.double())
    ref = linear(x, W, b, name, None, dY)
    assert torch.allclose(ref["Y"][0], y.detach()) and (name is None) == ("F" not in ref)
    for leaf, key in zip(leaves, ("dX", "dW", "dbias")):
        assert torch.allclose(ref[key][0], leaf.grad), key


def test_binding_refusals():
    x, W, ws = torch.zeros(4, 8).bfloat16(), torch.zeros(8, 16).bfloat16(), torch.zeros(1 << 20, dtype=torch.uint8)
    for call in (lambda: moe.moe_linear(x, W, ws=ws), lambda: moe.moe_linear(x, W), lambda: moe.moe_linear(x, W, act="tanh", ws=ws),
                 lambda: moe.moe_linear_train(x, W, ws=ws), lambda: moe.moe_linear_backward(x, x, W, None, ws=ws),
                 lambda: moe.linear_workspace(4, 12, 16)):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(TypeError):
        moe.moe_linear_backward(x, x, W, None, bias_dtype=torch.float64, ws=ws)
