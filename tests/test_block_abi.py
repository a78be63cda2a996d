"""The sub-block calls refuse bad arguments on the host, before the device is touched
(no GPU needed: a call that passes its checks stops at the architecture check)."""
import math

import pytest
import torch

from block_common import keep_mask, layernorm, layernorm_backward
from top_routing_grouped_02_gb300 import _build, moe

INVALID, SHAPE, SMALL = 1, 2, 3
P = 1 << 20  # an aligned address that is never read


@pytest.fixture(scope="module")
def lib():
    # the addresses are made up: a call that passed its checks would use them on a GPU
    if torch.cuda.is_available():
        pytest.skip("refusals are tested where there is no GPU")
    _build.build()
    return moe.lib()


def ln(lib, x=P, ldx=64, gamma=P, beta=P, T=4, d=64, eps=1e-5, t=0, wt=0, y=P, ldy=64, mean=P, rstd=P):
    return lib.moe_layernorm_forward(x, ldx, gamma, beta, T, d, eps, t, wt, y, ldy, mean, rstd, None)


def ln_bwd(lib, dy=P, lddy=64, x=P, ldx=64, gamma=P, mean=P, rstd=P, dres=None, lddres=0, T=4, d=64,
           t=0, wt=0, dx=P, lddx=64, dgamma=P, dbeta=P, scratch=P, nbytes=1 << 20):
    return lib.moe_layernorm_backward(dy, lddy, x, ldx, gamma, mean, rstd, dres, lddres, T, d, t, wt,
                                      dx, lddx, dgamma, dbeta, scratch, nbytes, None)


def drop(lib, x=P, ldx=64, res=None, ldr=0, T=4, d=64, p=0.1, ctr=None, t=0, y=P, ldy=64):
    return lib.moe_dropout(x, ldx, res, ldr, T, d, p, 1, 2, ctr, t, y, ldy, None)


def test_layernorm_refusals(lib):
    passed = ln(lib)
    assert passed not in (INVALID, SHAPE, SMALL)
    for bad in (dict(x=None), dict(y=None), dict(d=0), dict(T=-1), dict(eps=-1.0), dict(eps=math.nan),
                dict(t=3), dict(wt=1), dict(t=1, wt=0), dict(ldx=63), dict(ldy=63), dict(x=P + 1),
                dict(gamma=P + 1), dict(wt=2, gamma=P + 2), dict(mean=P + 2), dict(y=P, ldx=65)):
        assert ln(lib, **bad) == INVALID, bad
    assert ln(lib, ldx=1 << 57) == SHAPE
    assert ln(lib, T=0, x=None, y=None) == 0
    assert ln(lib, T=1, ldx=0) == passed  # a single row has no stride


def test_layernorm_backward_refusals(lib):
    passed = ln_bwd(lib)
    assert passed not in (INVALID, SHAPE, SMALL)
    for bad in (dict(dy=None), dict(x=None), dict(dx=None), dict(mean=None), dict(rstd=None),
                dict(lddy=3), dict(dres=P, lddres=63), dict(scratch=None), dict(scratch=P + 8),
                dict(wt=1), dict(t=7), dict(d=-4), dict(dgamma=P + 1)):
        assert ln_bwd(lib, **bad) == INVALID, bad
    assert ln_bwd(lib, nbytes=lib.moe_layernorm_scratch_bytes(4, 64) - 1) == SMALL
    assert ln_bwd(lib, dgamma=None, dbeta=None, scratch=None, nbytes=0) == passed
    assert lib.moe_layernorm_scratch_bytes(4, 0) == 0
    assert lib.moe_layernorm_scratch_bytes(1 << 20, 4096) <= 256 * 2 * 4 * 4096


def test_dropout_refusals(lib):
    passed = drop(lib)
    assert passed not in (INVALID, SHAPE, SMALL)
    for bad in (dict(x=None), dict(y=None), dict(p=-0.1), dict(p=1.1), dict(p=math.nan), dict(t=-1),
                dict(ldx=1), dict(res=P, ldr=5), dict(ctr=P + 4), dict(x=P + 1), dict(d=0), dict(T=-2)):
        assert drop(lib, **bad) == INVALID, bad
    assert drop(lib, T=1 << 56, d=64) == SHAPE
    assert drop(lib, T=0, x=None, y=None) == 0
    assert lib.moe_dropout_backward(None, 64, 4, 64, 0.1, 1, 2, None, 0, P, 64, None) == INVALID


def test_binding_refusals():
    cpu = torch.zeros(4, 8)
    for call in (lambda: moe.moe_layernorm(cpu), lambda: moe.moe_dropout(cpu, 0.1, 1),
                 lambda: moe.moe_dropout_backward(cpu, 0.1, 1),
                 lambda: moe.moe_layernorm_backward(cpu, cpu, None, cpu[:, 0], cpu[:, 0])):
        with pytest.raises(ValueError):
            call()


def test_philox_known_answers():
    # the published test vectors of Philox 4x32-10 with all-zero and all-one input:
    # counter and key 0 start with the words 6627e8d5 e169c58d bc57ac4c 9b00dbd8
    words = [0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8]
    halves = [h for w in words for h in (w & 0xFFFF, w >> 16)]
    for p in (0.1, 0.5, 0.9):
        thr = math.floor(p * 65536 + 0.5)
        assert keep_mask(8, p, 0, 0).tolist() == [h >= thr for h in halves]


def test_plain_backward_against_autograd():
    g = torch.Generator().manual_seed(0)
    x, dy = (torch.randn(5, 12, generator=g, dtype=torch.float64) for _ in range(2))
    gamma = torch.randn(12, generator=g, dtype=torch.float64)
    xa, ga = x.clone().requires_grad_(), gamma.clone().requires_grad_()
    (layernorm(xa, ga, None, 1e-5)[0] * dy).sum().backward()
    dx, dgamma, dbeta = layernorm_backward(dy, x, gamma, 1e-5)
    torch.testing.assert_close(dx, xa.grad)
    torch.testing.assert_close(dgamma, ga.grad)
    torch.testing.assert_close(dbeta, dy.sum(0))
