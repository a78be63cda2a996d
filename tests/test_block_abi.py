"""The sub-block calls refuse bad arguments on the host, before the device is touched
(no GPU needed: a call that passes its checks stops at the architecture check)."""
import math

import pytest
import torch

from block_common import ffn, keep_mask, layernorm, layernorm_backward
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
    assert lib.moe_layernorm_scratch_bytes(1 << 20, 4096) <= 384 * 2 * 4 * 4096


def test_dropout_refusals(lib):
    passed = drop(lib)
    assert passed not in (INVALID, SHAPE, SMALL)
    for bad in (dict(x=None), dict(y=None), dict(p=-0.1), dict(p=1.1), dict(p=math.nan), dict(t=-1),
                dict(ldx=1), dict(res=P, ldr=5), dict(ctr=P + 4), dict(x=P + 1), dict(d=0), dict(T=-2)):
        assert drop(lib, **bad) == INVALID, bad
    assert drop(lib, T=1 << 56, d=64) == SHAPE
    assert drop(lib, T=0, x=None, y=None) == 0
    assert lib.moe_dropout_backward(None, 64, 4, 64, 0.1, 1, 2, None, 0, P, 64, None) == INVALID


def ffn_fwd(lib, X=P, W1=P, W3=P, W2=P, T=4, d=64, n=128, act=0, t=0, Y=P, ws=P, nbytes=1 << 40):
    return lib.moe_ffn_forward(X, W1, W3, W2, T, d, n, act, t, Y, ws, nbytes, None)


def ffn_train(lib, T=4, d=64, n=128, H=P, A1=P, A3=P, ws=P, nbytes=1 << 40):
    return lib.moe_ffn_forward_train(P, P, P, P, T, d, n, 0, 0, P, H, A1, A3, ws, nbytes, None)


def ffn_bwd(lib, dY=P, A1=P, T=4, d=64, n=128, act=0, t=0, dX=P, dW1=P, dW3=P, dW2=P, ws=P, nbytes=1 << 40):
    return lib.moe_ffn_backward(dY, P, P, P, P, P, A1, P, T, d, n, act, t, dX, dW1, dW3, dW2, ws, nbytes, None)


def test_ffn_refusals(lib):
    passed = ffn_fwd(lib)
    assert passed not in (INVALID, SHAPE, SMALL)
    for bad in (dict(X=None), dict(W1=None), dict(W3=P + 8), dict(W2=None), dict(Y=None), dict(T=-1),
                dict(d=0), dict(n=-8), dict(act=2), dict(t=5), dict(ws=None), dict(ws=P + 16)):
        assert ffn_fwd(lib, **bad) == INVALID, bad
    for bad in (dict(d=12), dict(n=4), dict(t=2), dict(d=(1 << 20) + 8)):
        assert ffn_fwd(lib, **bad) == SHAPE, bad
    for T in (1, 128, 129):
        need = lib.moe_ffn_workspace_bytes(T, 64, 128, 0)
        assert ffn_fwd(lib, T=T, nbytes=need - 1) == SMALL
        assert ffn_fwd(lib, T=T, nbytes=need) == passed
        assert lib.moe_ffn_workspace_bytes(T, 64, 128, 1) >= need
    assert ffn_fwd(lib, T=0, X=None) == 0
    assert ffn_train(lib) == passed
    for bad in (dict(H=None), dict(A1=None), dict(A3=P + 4)):
        assert ffn_train(lib, **bad) == INVALID, bad
    assert ffn_bwd(lib) == passed
    assert ffn_bwd(lib, dX=None) == passed
    assert ffn_bwd(lib, dW1=None, dW3=None, dW2=None) == passed
    for bad in (dict(dY=None), dict(A1=None), dict(dX=P + 8), dict(dW1=None), dict(dW2=None),
                dict(dW3=P + 2), dict(act=-1), dict(ws=None)):
        assert ffn_bwd(lib, **bad) == INVALID, bad
    assert ffn_bwd(lib, T=300, nbytes=lib.moe_ffn_workspace_bytes(300, 64, 128, 1) - 1) == SMALL
    assert lib.moe_ffn_workspace_bytes(4, 60, 128, 0) == 0
    assert lib.moe_ffn_workspace_init(P, 64, None) == SMALL


def test_plain_ffn_against_autograd():
    g = torch.Generator().manual_seed(1)
    for act in ("silu", "gelu"):
        x, W1, W3 = (torch.randn(*s, generator=g).bfloat16() for s in ((5, 12), (12, 9), (12, 9)))
        W2, dY = torch.randn(9, 12, generator=g).bfloat16(), torch.randn(5, 12, generator=g).bfloat16()
        leaves = [t.double().requires_grad_() for t in (x, W1, W3, W2)]
        f = torch.nn.functional.silu if act == "silu" else lambda a: torch.nn.functional.gelu(a, approximate="tanh")
        y = (f(leaves[0] @ leaves[1]) * (leaves[0] @ leaves[2])) @ leaves[3]
        y.backward(dY.double())
        ref = ffn(x, W1, W3, W2, act, dY)
        for name, want in zip(("Y", "dX", "dW1", "dW3", "dW2"), [y.detach()] + [t.grad for t in leaves]):
            torch.testing.assert_close(ref[name][0], want)


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
