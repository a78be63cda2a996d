"""Projections whose outputs lie on operands or on one another are refused on the host: tiles would be
overwritten while others still read them."""
import pytest

from test_linear_abi import A, INVALID, SHAPE, SMALL, bwd, fwd, lib, train  # noqa: F401

T, K, N = 4, 64, 128
X, W, BIAS, RES, Y, F, WS, DX, DW, DB = A[:10]
# bytes of each at these sizes (F in blocks of 32 x 32 fp32)
SIZE = {"X": T * K * 2, "W": K * N * 2, "b": N * 2, "r": T * N * 2, "Y": T * N * 2, "F": 32 * N * 4, "dX": T * K * 2,
        "dW": K * N * 2, "db": N * 2, "dY": T * N * 2}


def refused(call, lib, out, at, size):  # noqa: F811
    """`out` over, at the end of and in front of the operand's bytes: refused; next to them: not."""
    ok = call(lib)
    assert ok not in (INVALID, SHAPE, SMALL)
    for over in (at, at + size - 16, at - SIZE[out] + 16):
        assert call(lib, **{out: over}) == INVALID, (out, at, over)
    for beside in (at + size, at - SIZE[out]):
        assert call(lib, **{out: beside}) == ok, (out, at, beside)


def test_forward(lib):  # noqa: F811
    for call in (fwd, train):
        for at, name in ((X, "X"), (W, "W"), (BIAS, "b")):
            refused(call, lib, "Y", at, SIZE[name])
        # in the residual's place, or off it
        ok = call(lib)
        assert call(lib, Y=RES) == ok
        for off in (16, -16, SIZE["r"] - 16):
            assert call(lib, Y=RES + off) == INVALID, off
    for at, name in ((X, "X"), (W, "W"), (BIAS, "b"), (RES, "r"), (Y, "Y")):
        refused(train, lib, "F", at, SIZE[name])


def test_fp32_bias(lib):  # noqa: F811
    """The bias' own type counts: 4 bytes an element."""
    assert fwd(lib, bt=2, Y=BIAS + N * 2) == INVALID and fwd(lib, bt=2, Y=BIAS + N * 4) == fwd(lib)
    assert bwd(lib, bt=2, dX=DB + N * 2) == INVALID and bwd(lib, bt=2, dX=DB + N * 4) == bwd(lib)


def test_backward(lib):  # noqa: F811
    for out in ("dX", "dW", "db"):
        for at, name in ((X, "X"), (W, "W"), (RES, "dY"), (F, "F")):
            refused(bwd, lib, out, at, SIZE[name])
        for other, at in (("dX", DX), ("dW", DW), ("db", DB)):
            if other != out:
                refused(bwd, lib, out, at, SIZE[other])


@pytest.mark.parametrize("call", [fwd, train, bwd])
def test_without_tokens_nothing_overlaps(lib, call):  # noqa: F811
    over = {fwd: dict(Y=W), train: dict(Y=W, F=W), bwd: dict(dX=W)}[call]
    assert call(lib, T=0, **over) == call(lib, T=0)
