"""Refusals of the norms around a block, and the plain gradients of their tests (no GPU needed)."""
import math

import pytest
import torch

import norms_common as plain
from top_routing_grouped_02_gb300 import _build, moe

INVALID, SHAPE, SMALL = 1, 2, 3
A = [(i + 1) << 24 for i in range(12)]  # aligned addresses that are never read
POST, PRE = 1, 2


@pytest.fixture(scope="module")
def lib():
    # the addresses are made up: a call that passed its checks would use them on a GPU
    if torch.cuda.is_available():
        pytest.skip("refusals are tested where there is no GPU")
    _build.build()
    return moe.lib()


def fwd(lib, x=A[0], ldx=64, b=A[1], ldb=64, gate=A[2], ldg=64, kind=2, post=A[3], pre=A[3], scale=1.0,
        norms=POST | PRE, T=4, d=64, eps=1e-6, t=0, wt=0, y=A[4], ldy=64, u=A[5], ldu=64, rp=A[6], rq=A[6]):
    return lib.moe_block_norm_forward(x, ldx, b, ldb, gate, ldg, kind, post, pre, scale, norms, T, d, eps, t, wt,
                                      y, ldy, u, ldu, rp, rq, None)


def bwd(lib, dy=A[7], lddy=64, du=A[8], lddu=64, x=A[0], ldx=64, b=A[1], ldb=64, gate=A[2], ldg=64, kind=2,
        post=A[3], pre=A[3], scale=1.0, norms=POST | PRE, rp=A[6], rq=A[6], T=4, d=64, t=0, wt=0, dx=A[4], lddx=64,
        db=A[5], lddb=64, dgate=A[9], lddg=64, dpost=A[10], dpre=A[10], scratch=A[11], nbytes=1 << 20):
    return lib.moe_block_norm_backward(dy, lddy, du, lddu, x, ldx, b, ldb, gate, ldg, kind, post, pre, scale, norms,
                                       rp, rq, T, d, t, wt, dx, lddx, db, lddb, dgate, lddg, dpost, dpre, scratch,
                                       nbytes, None)


COMMON = [dict(x=None), dict(x=A[0] + 1), dict(b=None), dict(gate=None), dict(kind=3), dict(kind=0), dict(norms=4),
          dict(T=-1), dict(d=0), dict(t=3), dict(t=1, wt=0), dict(wt=2, post=A[3] + 2), dict(pre=A[3] + 1),
          dict(ldx=63), dict(ldb=63), dict(ldg=63), dict(scale=math.nan), dict(kind=1, gate=A[2] + 2),
          dict(norms=POST), dict(rp=A[6] + 2), dict(rq=A[6] + 1)]


def test_forward_refusals(lib):
    assert fwd(lib) not in (INVALID, SHAPE)
    for bad in COMMON + [dict(y=None), dict(u=None), dict(y=A[5]), dict(ldy=63), dict(y=A[0], ldy=65), dict(u=A[1], ldu=65),
                         dict(y=A[2], ldy=72), dict(eps=-1.0), dict(eps=math.nan)]:
        assert fwd(lib, **bad) == INVALID, bad
    assert fwd(lib, d=16385, ldx=16385) == SHAPE and fwd(lib, ldx=1 << 57) == SHAPE and fwd(lib, T=1 << 55) == SHAPE
    assert fwd(lib, T=0, x=None, b=None, y=None, u=None) == 0
    ok = fwd(lib)
    for good in (dict(kind=0, gate=None), dict(kind=1), dict(norms=POST, pre=None, u=None), dict(norms=0, pre=None, u=None),
                 dict(y=A[0]), dict(u=A[2]), dict(rp=None, rq=None), dict(post=None, pre=None), dict(wt=2)):
        assert fwd(lib, **good) == ok, good
    rms = dict(b=None, y=None, gate=None, kind=0, post=None, norms=PRE)
    assert fwd(lib, **rms) == ok
    for bad in (dict(y=A[4]), dict(kind=1, gate=A[2]), dict(post=A[3]), dict(norms=POST | PRE), dict(norms=0, pre=None, u=None),
                dict(scale=2.0), dict(u=None)):
        assert fwd(lib, **(rms | bad)) == INVALID, bad


def test_backward_refusals(lib):
    ok = bwd(lib)
    assert ok not in (INVALID, SHAPE, SMALL)
    for bad in COMMON + [dict(du=None), dict(dx=None), dict(db=None), dict(dgate=None), dict(rp=None), dict(rq=None),
                         dict(dx=A[5]), dict(dgate=A[4]), dict(lddx=63), dict(lddg=63), dict(dx=A[7], lddx=72),
                         dict(db=A[0], lddb=72), dict(dgate=A[2], lddg=72), dict(scratch=None), dict(scratch=A[11] + 128),
                         dict(dpost=A[10] + 1), dict(kind=1, dgate=A[9] + 2),
                         dict(norms=POST, pre=None, du=None, dpre=None, dy=None), dict(norms=POST, pre=None, dpre=None),
                         dict(norms=POST, pre=None, du=None)]:
        assert bwd(lib, **bad) == INVALID, bad
    assert bwd(lib, nbytes=0) == SMALL and bwd(lib, d=16385) == SHAPE
    for good in (dict(dy=None), dict(dx=A[7]), dict(db=A[1], dx=A[0], dgate=A[2]), dict(dpost=None, dpre=None, scratch=None),
                 dict(norms=PRE, rp=None), dict(norms=POST, pre=None, du=None, dpre=None), dict(kind=0, gate=None, dgate=None)):
        assert bwd(lib, **good) == ok, good
    rms = dict(b=None, db=None, gate=None, dgate=None, kind=0, post=None, dpost=None, norms=PRE)
    assert bwd(lib, **rms) == ok
    for bad in (dict(db=A[5]), dict(dpost=A[10]), dict(dgate=A[9]), dict(scale=0.5)):
        assert bwd(lib, **(rms | bad)) == INVALID, bad


@pytest.mark.parametrize("gate", [None, "row", "full"])
@pytest.mark.parametrize("norms", [(1, 1), (1, 0), (0, 1), (0, 0)])
def test_plain_gradients(gate, norms):
    """The plain gradients that the GPU tests compare with, against autograd."""
    gen = torch.Generator().manual_seed(3)
    T, d, eps, scale = 5, 9, 1e-2, 0.5
    v = {k: torch.randn(T, d, generator=gen).double() for k in ("x", "b")}
    v |= {k: torch.randn(d, generator=gen).double() for k in ("post", "pre")}
    if gate is not None:
        v["gate"] = torch.randn((T, d) if gate == "full" else (T,), generator=gen).double()
    dy, du = (torch.randn(T, d, generator=gen).double() for _ in range(2))
    for t in v.values():
        t.requires_grad_()
    args = (v["x"], v["b"], v["post"], v["pre"], v.get("gate"), scale, eps, *norms)
    o = plain.forward(*args)
    loss = (o["y"] * dy).sum() + ((o["u"] * du).sum() if norms[1] else 0)
    loss.backward()
    with torch.no_grad():
        ref = plain.backward(dy, du, *args)
    for name, (value, size) in ref.items():
        assert torch.allclose(value, v[name[1:]].grad), name
        assert (size * (1 + 1e-12) >= value.abs()).all(), name
    assert ("dpre" in ref) == bool(norms[1]) and ("dgate" in ref) == (gate is not None)


def test_binding_refusals():
    x, w = torch.zeros(4, 8), torch.zeros(4)
    for call in (lambda: moe.moe_block_norm(x, x), lambda: moe.moe_rmsnorm(x),
                 lambda: moe.moe_block_norm_backward(x, x, x, x, None, None, w, w),
                 lambda: moe.moe_rmsnorm_backward(x, x, None, w)):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: moe.moe_block_norm(x, None), lambda: moe.moe_rmsnorm_backward(None, x, None, w),
                 lambda: moe.moe_block_norm_backward(x, x, x, x, None, None, w, w, wdtype=torch.float64)):
        with pytest.raises(TypeError):
            call()
