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


def keep_mask(n, p, seed, offset, first=0):
    """[n] bool: the definition of the dropout mask for elements first .. first + n - 1
    (first a multiple of 8), in Python integers."""
    thr = math.floor(p * 65536 + 0.5)
    out = []
    for block in range(first // 8, first // 8 + (n + 7) // 8):
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


def _act(a, act):
    """The activation, its derivative (64 bits)."""
    if act == "silu":
        sg = torch.sigmoid(a)
        return a * sg, sg * (1 + a * (1 - sg))
    c = math.sqrt(2 / math.pi)
    t = torch.tanh(c * (a + 0.044715 * a ** 3))
    return 0.5 * a * (1 + t), 0.5 * (1 + t) + 0.5 * a * (1 - t * t) * c * (1 + 3 * 0.044715 * a * a)


def ffn(x, W1, W3, W2, act, dY=None):
    """{name: (value, slack)}: the block's outputs in 64 bits, and for each element a
    bound on the error in front of its final rounding. Counted: one rounding (u) of
    H, dA1 and dA3 to 16 bits, K accumulations of at most 2^-23 of the sum of
    absolute terms each, and 2^-19 for the activation's approximate exponential and
    division. |act'| <= 1.2 and |act''| <= 1.2."""
    u, e32 = HALF[x.dtype], 2.0 ** -23
    x, W1, W3, W2 = (t.double() for t in (x, W1, W3, W2))
    d, n = W1.shape
    a1, a3 = x @ W1, x @ W3
    e1, e3 = (d * e32 * (x.abs() @ w.abs()) for w in (W1, W3))
    f, df = _act(a1, act)
    H = f * a3
    eH = 1.2 * e1 * (a3.abs() + e3) + f.abs() * e3 + 2.0 ** -19 * H.abs()
    eH = eH + u * (H.abs() + eH)
    out = {"Y": (H @ W2, eH @ W2.abs() + n * e32 * ((H.abs() + eH) @ W2.abs()))}
    if dY is None:
        return out
    dY = dY.double()
    T = x.shape[0]
    G, eG = dY @ W2.T, d * e32 * (dY.abs() @ W2.abs().T)
    dA1, dA3 = G * a3 * df, G * f
    eA1 = eG * (a3 * df).abs() + (G.abs() + eG) * (1.2 * e3 + 1.2 * a3.abs() * e1) + 2.0 ** -19 * (G * a3).abs()
    eA3 = eG * f.abs() + (G.abs() + eG) * 1.2 * e1 + 2.0 ** -19 * dA3.abs()
    eA1, eA3 = eA1 + u * (dA1.abs() + eA1), eA3 + u * (dA3.abs() + eA3)
    xa, ya = x.abs(), dY.abs()
    b1, b3 = dA1.abs() + eA1, dA3.abs() + eA3
    out["dX"] = (dA1 @ W1.T + dA3 @ W3.T, eA1 @ W1.abs().T + eA3 @ W3.abs().T
                 + 2 * n * e32 * (b1 @ W1.abs().T + b3 @ W3.abs().T))
    out["dW1"] = (x.T @ dA1, xa.T @ eA1 + T * e32 * (xa.T @ b1))
    out["dW3"] = (x.T @ dA3, xa.T @ eA3 + T * e32 * (xa.T @ b3))
    out["dW2"] = (H.T @ dY, eH.T @ ya + T * e32 * ((H.abs() + eH).T @ ya))
    return out


def check_ffn(got, ref, name):
    """Every element within its bound, and the whole within 1.5 u in the 2-norm (two
    independent roundings of at most u each give sqrt(2) u)."""
    want, slack = ref
    u = HALF[got.dtype]
    g = got.double()
    assert torch.isfinite(g).all(), f"{name}: not finite"
    bound = u * (want.abs() + slack) + slack + TINY[got.dtype]
    err = (g - want).abs()
    assert (err <= bound).all(), f"{name}: worst {float((err / bound).max()):.3f} of its bound"
    if want.numel() >= 64:  # a norm over a few elements says no more than they do
        rel = float(err.norm() / want.norm())
        assert rel <= 1.5 * u, f"{name}: 2-norm error {rel:.2e} of u {u:.2e}"
