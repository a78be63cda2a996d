"""Refusals of the calls that move rows between token order and expert order (no GPU needed)."""
import pytest
import torch

import rows_common as plain
from top_routing_grouped_02_gb300 import _build, moe

INVALID, SHAPE = 1, 2
P, Q, S = 1 << 20, 1 << 24, 1 << 28  # aligned addresses that are never read


@pytest.fixture(scope="module")
def lib():
    # the addresses are made up: a call that passed its checks would use them on a GPU
    if torch.cuda.is_available():
        pytest.skip("refusals are tested where there is no GPU")
    _build.build()
    return moe.lib()


def dispatch(lib, x=P, ldx=64, row=P, T=4, K=2, d=64, t=0, xg=Q, ldxg=64, rows=8):
    return lib.moe_dispatch(x, ldx, row, T, K, d, t, xg, ldxg, rows, None)


def combine(lib, z=P, ldz=64, rows=8, row=P, w=P, res=None, ldr=0, T=4, K=2, d=64, t=0, y=Q, ldy=64):
    return lib.moe_combine_weighted(z, ldz, rows, row, w, res, ldr, T, K, d, t, y, ldy, None)


def backward(lib, dy=P, lddy=64, z=Q, ldz=64, rows=8, row=P, w=P, T=4, K=2, d=64, t=0, dz=S, lddz=64, dw=P):
    return lib.moe_combine_weighted_backward(dy, lddy, z, ldz, rows, row, w, T, K, d, t, dz, lddz, dw, None)


COMMON = [dict(row=None), dict(row=P + 2), dict(T=-1), dict(K=0), dict(d=0), dict(t=3), dict(rows=-1)]
TOO_LARGE = [dict(K=9), dict(T=1 << 30, K=2), dict(T=1 << 60), dict(d=(1 << 28) + 1, ldx=1 << 29, ldz=1 << 29, ldy=1 << 29, lddy=1 << 29)]


@pytest.mark.parametrize("call,bad", [
    (dispatch, [dict(x=None), dict(xg=None), dict(x=P + 1), dict(xg=Q + 1), dict(t=2, x=P + 2), dict(ldx=63),
                dict(ldxg=63), dict(xg=P)]),
    (combine, [dict(z=None), dict(y=None), dict(z=P + 1), dict(y=Q + 1), dict(w=P + 2), dict(ldz=63), dict(ldy=63),
               dict(y=P), dict(res=S + 1, ldr=64), dict(res=S, ldr=63), dict(res=Q, ldr=65)]),
    (backward, [dict(dy=None), dict(z=None), dict(dz=None), dict(w=None), dict(dw=None), dict(dw=P + 2),
                dict(w=P + 1), dict(lddy=63), dict(ldz=63), dict(lddz=63), dict(dz=P), dict(dz=Q, lddz=65)]),
], ids=["dispatch", "combine", "backward"])
def test_refusals(lib, call, bad):
    assert call(lib) not in (INVALID, SHAPE)
    for b in COMMON + bad:
        assert call(lib, **b) == INVALID, b
    for b in TOO_LARGE:
        b = {k: v for k, v in b.items() if k in call.__code__.co_varnames}
        assert call(lib, **b) == SHAPE, b
    assert call(lib, T=0) == 0


def test_plain_gradients():
    """The plain gradients that the GPU tests compare with, against autograd."""
    gen = torch.Generator().manual_seed(5)
    T, K, d = 7, 3, 5
    row, used = plain.slot_map(T, K, 4, 0.2, gen)
    z, w, dy = (torch.randn(*s, generator=gen, dtype=torch.float64) for s in ((T * K, d), (T, K), (T, d)))
    z.requires_grad_(), w.requires_grad_()
    y, _ = plain.combine(z, row, w)
    y.backward(dy)
    dz, dw, _ = plain.combine_backward(dy, z.detach(), row, w.detach(), torch.zeros(T * K, d))
    assert torch.allclose(dz, z.grad) and torch.allclose(dw, w.grad) and not dz[used:].any()
    x = torch.randn(T, d, generator=gen, dtype=torch.float64)
    xg = plain.dispatch(x, row, K, torch.zeros(T * K, d))
    dx, _ = plain.combine(z.detach(), row, K)
    assert torch.allclose((xg * z.detach()).sum(), (x * dx).sum())


def test_binding_refusals():
    """What the Python side refuses before the library is called: tensors on the CPU."""
    x, row = torch.zeros(4, 8), torch.zeros(8, dtype=torch.int32)
    for call in (lambda: moe.moe_dispatch(x, row, 2), lambda: moe.moe_dispatch_backward(x, row, 2),
                 lambda: moe.moe_combine_weighted(x, row, torch.zeros(4, 2)),
                 lambda: moe.moe_combine_weighted_backward(x, x, row, torch.zeros(4, 2))):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(TypeError):
        moe.moe_combine_weighted(x, row, 2)
    with pytest.raises(ValueError):
        moe.moe_combine_weighted(x, row, torch.zeros(8))
