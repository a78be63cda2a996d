"""Plain 64-bit forms of the sub-block operators and the tolerances of their tests.

A result rounded once to a type of p-bit precision is off by at most half a step,
eps / 2 relative to its value (torch.finfo: bf16 2^-8, fp16 2^-11, fp32 2^-24).
fp32 arithmetic in front of it adds an error that is bounded per operator by the
sums it takes; each test states it as a multiple of 2^-24 times the terms' size.
"""
import math

import torch

HALF = {t: torch.finfo(t).eps / 2 for t in (torch.bfloat16, torch.float16, torch.float32)}
# smallest spacing near zero: half of it is the error of a result that underflows
TINY = {torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25, torch.float32: 2.0 ** -150}
U32 = 2.0 ** -24


def assert_close(got, want, terms, c, what):
    """|got - want| <= rounding of `want` + c * 2^-24 * terms (64-bit tensors)."""
    g = got.double().cpu()
    w = want.double().cpu()
    tm = terms.double().cpu() if torch.is_tensor(terms) else torch.full_like(w, float(terms))
    slack = c * U32 * tm
    bound = HALF[got.dtype] * (w.abs() + slack) + slack + TINY[got.dtype]
    err = (g - w).abs()
    assert torch.isfinite(g).all(), f"{what}: not finite"
    bad = err > bound
    assert not bad.any(), (f"{what}: {int(bad.sum())} of {bad.numel()} off, worst "
                           f"{float((err / bound).max()):.3f} of its bound")


def layernorm(x, gamma, beta, eps):
    """(y, mean, rstd, xhat) in 64 bits."""
    x = x.double()
    mean = x.mean(-1, keepdim=True)
    c = x - mean
    rstd = 1 / torch.sqrt((c * c).mean(-1, keepdim=True) + eps)
    xh = c * rstd
    y = xh if gamma is None else xh * gamma.double()
    return (y if beta is None else y + beta.double()), mean, rstd, xh


def layernorm_backward(dy, x, gamma, eps, dres=None):
    dy = dy.double()
    _, _, rstd, xh = layernorm(x, None, None, eps)
    g = dy if gamma is None else dy * gamma.double()
    dx = rstd * (g - g.mean(-1, keepdim=True) - xh * (g * xh).mean(-1, keepdim=True))
    return (dx if dres is None else dx + dres.double()), (dy * xh).sum(0), dy.sum(0)


def keep_mask(n, p, seed, offset):
    """[n] bool: the definition of the dropout mask, in Python integers."""
    thr = math.floor(p * 65536 + 0.5)
    out = []
    for block in range((n + 7) // 8):
        c = [block & 0xFFFFFFFF, block >> 32, offset & 0xFFFFFFFF, offset >> 32]
        k = [seed & 0xFFFFFFFF, seed >> 32]
        for _ in range(10):
            a, b = c[0] * 0xD2511F53, c[2] * 0xCD9E8D57
            c = [(b >> 32) ^ c[1] ^ k[0], b & 0xFFFFFFFF, (a >> 32) ^ c[3] ^ k[1], a & 0xFFFFFFFF]
            k = [(k[0] + 0x9E3779B9) & 0xFFFFFFFF, (k[1] + 0xBB67AE85) & 0xFFFFFFFF]
        for w in c:
            out += [(w & 0xFFFF) >= thr, (w >> 16) >= thr]
    return torch.tensor(out[:n], dtype=torch.bool)


def dropout_scale(p):
    thr = math.floor(p * 65536 + 0.5)
    return 65536 / (65536 - thr) if thr < 65536 else 0.0


def matrix(T, d, dtype, gen, ld=None, scale=1.0, shift=0.0, device="cuda"):
    """[T, d] view of a [T, ld] buffer of normal values."""
    v = torch.randn(max(T, 1), ld or d, generator=gen, dtype=torch.float64) * scale + shift
    return v.to(dtype).to(device)[:T, :d]
