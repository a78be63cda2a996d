"""An output in the place of an operand has to have its row stride: with another one, rows
would be overwritten before they are read. Refused on the host, before the device is touched."""
import pytest
import torch

from top_routing_grouped_02_gb300 import _build, moe

INVALID = 1
P, Q, R, S = ((k + 1) << 20 for k in range(4))  # aligned addresses that are never read


@pytest.fixture(scope="module")
def lib():
    if torch.cuda.is_available():
        pytest.skip("refusals are tested where there is no GPU: the addresses are made up")
    _build.build()
    return moe.lib()


def ln_bwd(lib, dy=P, lddy=64, x=Q, ldx=64, dres=R, lddres=64, dx=S, lddx=64, T=4):
    return lib.moe_layernorm_backward(dy, lddy, x, ldx, P, P, P, dres, lddres, T, 64, 0, 0, dx, lddx, P, P, P, 1 << 20,
                                      None)


def drop(lib, x=P, ldx=64, res=Q, ldr=64, y=R, ldy=64, T=4):
    return lib.moe_dropout(x, ldx, res, ldr, T, 64, 0.1, 1, 2, None, 0, y, ldy, None)


def drop_bwd(lib, dy=P, lddy=64, dx=R, lddx=64, T=4):
    return lib.moe_dropout_backward(dy, lddy, T, 64, 0.1, 1, 2, None, 0, dx, lddx, None)


@pytest.mark.parametrize("call,operands,out", [
    (ln_bwd, (("dy", "lddy", P), ("x", "ldx", Q), ("dres", "lddres", R)), ("dx", "lddx")),
    (drop, (("x", "ldx", P), ("res", "ldr", Q)), ("y", "ldy")),
    (drop_bwd, (("dy", "lddy", P),), ("dx", "lddx"))])
def test_output_over_an_operand(lib, call, operands, out):
    passed = call(lib)
    assert passed not in (1, 2, 3)
    for name, ld, at in operands:
        over = {out[0]: at}
        assert call(lib, **over) == passed, name
        assert call(lib, **over, **{out[1]: 72, ld: 72}) == passed, name
        for other in ({out[1]: 72}, {ld: 72}):
            assert call(lib, **over, **other) == INVALID, (name, other)
            assert call(lib, **over, **other, T=1) == passed  # a single row has no stride
            assert call(lib, **other) == passed
