"""A projection with its epilogue in 64 bits, and what each element may be off by in front of
its final rounding.

Counted: a sum of K products accumulated in fp32 is off by at most K 2^-23 of its absolute terms
(the tensor cores may truncate), the bias' and the residual's sums by 2^-24 of what they give,
the activation by its slope (|act'| <= 1.2, |act''| <= 1.2) and 2^-19 for its approximate
exponential and division. dA = dY F, F = act'(A) in fp32, is rounded to 16 bits (u) as an
operand of the products, and not for dbias."""
import torch

from block_common import HALF, _act

E32 = 2.0 ** -23


def act(a, name):
    return (a, torch.ones_like(a)) if name is None else _act(a, name)


def linear(x, W, bias, name, res, dY=None):
    """{name: (value, slack)} of Y, F and, with dY, dX, dW and dbias."""
    u = HALF[x.dtype]
    x, W = x.double(), W.double()
    T, (k, n) = x.shape[0], W.shape
    a = x @ W
    ea = k * E32 * (x.abs() @ W.abs())
    if bias is not None:
        a = a + bias.double()
    ea = ea + E32 * a.abs()
    f, df = act(a, name)
    slope, curve, approx = (1.0, 0.0, 0.0) if name is None else (1.2, 1.2, 2.0 ** -19)
    Y, eY = f, slope * ea + approx * (a.abs() + f.abs())
    if res is not None:
        Y = Y + res.double()
        eY = eY + E32 * Y.abs()
    out = {"Y": (Y, eY)}
    eF = curve * ea + approx * (1 + a.abs())
    if name is not None:
        out["F"] = (df, eF)
    if dY is None:
        return out
    dY = dY.double()
    eF = eF * (name is not None)
    dA, eA = dY * df, dY.abs() * (eF + E32 * df.abs())
    A = dA.abs() + eA
    out["dbias"] = (dA.sum(0), eA.sum(0) + T * E32 * A.sum(0))
    if name is not None:
        eA = eA + u * A + 2.0 ** -25
        A = dA.abs() + eA
    out["dX"] = (dA @ W.T, eA @ W.abs().T + n * E32 * (A @ W.abs().T))
    out["dW"] = (x.T @ dA, x.abs().T @ eA + T * E32 * (x.abs().T @ A))
    return out
