"""The operators around the expert GEMMs of a transformer's feed-forward sub-block, as cases to measure.

  layernorm   the norm in front of the router and the experts, forward and backward (with the weight
              gradients' reduction over all rows and, as the residual stream needs it, the other
              branch's gradient added in)
  dropout     residual + dropout(x) behind them, from a counter-based generator: the mask is a function of
              (seed, offset, element) and is never stored; its backward is the same function of dy
  ffn         the dense gated feed-forward block (a shared expert, or a layer without experts):
              Y = (act(X W1) * (X W3)) W2, forward, and forward with backward

`own` chooses between the plain form below (elementary torch operations in 32 bits) and this framework's calls.
"""
import math

import numpy as np
import torch

own = False

_TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
_EPS = 1e-5


# --------------------------------------------------------------------------- cases


def _ln(T, d, dtype, wdtype, train, dres=False, ld=0):
    return {"op": "layernorm", "T": T, "d": d, "dtype": dtype, "wdtype": wdtype, "train": train, "dres": dres, "ld": ld or d}


def _dp(T, d, dtype, p, residual, train, ld=0):
    return {"op": "dropout", "T": T, "d": d, "dtype": dtype, "p": p, "residual": residual, "train": train, "ld": ld or d}


def _ff(T, d, n, dtype, act, train):
    return {"op": "ffn", "T": T, "d": d, "n": n, "dtype": dtype, "act": act, "train": train}


def listed():
    return [
        # one new token in front of the router, at the width of the Mixtral-shaped layer: latency alone
        dict(_ln(1, 4096, "bf16", "bf16", False), name="ln_one_token"),
        # a training step's norm at the Mixtral-shaped layer, parameters kept in 32 bits
        dict(_ln(4096, 4096, "bf16", "fp32", True), name="ln_train_4096x4096"),
        # the same at the widest layer, with the residual branch's gradient added
        dict(_ln(8192, 7168, "bf16", "bf16", True, dres=True), name="ln_train_8192x7168"),
        # an odd width in 32 bits: no row but the first starts on a 16-byte boundary
        dict(_ln(1537, 1023, "fp32", "fp32", True), name="ln_train_odd_fp32"),
        # residual dropout of a short batch: latency
        dict(_dp(64, 1536, "bf16", 0.1, True, False), name="drop_64x1536"),
        # a training step's residual dropout at the SonicMoE-shaped layer, both directions
        dict(_dp(16384, 1536, "bf16", 0.1, True, True), name="drop_train_16384x1536"),
        # rows that lie in a wider buffer, an odd length, 32 bits, no residual
        dict(_dp(1023, 2047, "fp32", 0.25, False, True, ld=2050), name="drop_train_strided_fp32"),
        # one new token through a dense block of the Mixtral-shaped expert's size: the weights are streamed
        dict(_ff(1, 4096, 14336, "bf16", "silu", False), name="ffn_one_token"),
        # a batch of 48 decoding sequences through a shared expert of the DeepSeek-V3-shaped layer, 16-bit floats
        dict(_ff(48, 7168, 2048, "fp16", "gelu", False), name="ffn_48_tokens_fp16"),
        # a short prompt through the same block
        dict(_ff(512, 7168, 2048, "bf16", "silu", False), name="ffn_512_tokens"),
        # a training step with ragged sizes: no dimension is a multiple of a tile
        dict(_ff(777, 1000, 2728, "bf16", "gelu", True), name="ffn_train_ragged"),
        # a training step of the Mixtral-shaped expert as a dense block: the largest
        dict(_ff(4096, 4096, 14336, "bf16", "silu", True), name="ffn_train_4096"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["layernorm", "dropout", "ffn"])
    train = rng.random() < 0.6
    if op == "ffn":
        # widths in steps of 8, as the call takes them; any number of tokens
        d, n = 8 * _log(rng, 16, 896), 8 * _log(rng, 16, 1792)
        most = 4096 * 4096 * 14336 // (d * n)
        T = _log(rng, 64, min(8192, most)) if train else _log(rng, 1, 2048)
        return _ff(T, d, n, rng.choice(["bf16", "bf16", "fp16"]), rng.choice(["silu", "gelu"]), train)
    d = _log(rng, 64, 8192)
    if rng.random() < 0.6:
        d = (d + 7) // 8 * 8
    T = _log(rng, 1, min(16384, 8192 * 7168 // d))
    dtype = rng.choice(["bf16", "bf16", "fp16", "fp32"])
    ld = d + rng.choice([0, 0, 0, 8, 3])
    if op == "layernorm":
        return _ln(T, d, dtype, rng.choice([dtype, "fp32"]), train, train and rng.random() < 0.5, ld)
    return _dp(T, d, dtype, rng.choice([0.05, 0.1, 0.2, 0.5]), rng.random() < 0.6, train, ld)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    dt = _TYPES[case["dtype"]]

    def normal(*shape, scale=1.0, dtype=dt, shift=None):
        v = torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32).mul_(scale)
        return (v if shift is None else v.add_(shift)).to(dtype)

    s = {"case": dict(case)}
    T, d = case["T"], case["d"]
    if case["op"] == "ffn":
        n = case["n"]
        s |= {"x": normal(T, d), "w1": normal(d, n, scale=d**-0.5), "w3": normal(d, n, scale=d**-0.5), "w2": normal(n, d, scale=n**-0.5)}
        if case["train"]:
            s["dy"] = normal(T, d)
        if own:  # the scratch memory that a user's program keeps between calls
            from top_routing_grouped_02_gb300 import moe

            s["ws"] = moe.ffn_workspace(T, d, n, train=case["train"])
        return s
    ld = case["ld"]
    if case["op"] == "layernorm":
        # a residual stream: channels with offsets of their own, rows of different scale
        shift = normal(ld, dtype=torch.float32) * 0.5 + 1.0
        wdt = _TYPES[case["wdtype"]]
        s |= {"x": normal(T, ld, scale=2.0, shift=shift)[:, :d], "gamma": normal(d, scale=0.2, dtype=wdt, shift=1.0), "beta": normal(d, scale=0.2, dtype=wdt)}
    else:
        s |= {"x": normal(T, ld)[:, :d], "seed": 0x9E3779B97F4A7C15 ^ int(seed), "offset": 1000 + int(seed) % 1000}
        if case["residual"]:
            s["res"] = normal(T, ld, scale=2.0)[:, :d]
    if case["train"]:
        s["dy"] = normal(T, ld)[:, :d]
    if case.get("dres"):
        s["dres"] = normal(T, ld)[:, :d]
    return s


# --------------------------------------------------------------------------- one pass


def run(s):
    return {"layernorm": _run_layernorm, "dropout": _run_dropout, "ffn": _run_ffn}[s["case"]["op"]](s)


def _run_layernorm(s):
    c = s["case"]
    if own:
        from top_routing_grouped_02_gb300 import moe

        if not c["train"]:
            return {"y": moe.moe_layernorm(s["x"], s["gamma"], s["beta"], _EPS)}
        y, mean, rstd = moe.moe_layernorm(s["x"], s["gamma"], s["beta"], _EPS, stats=True)
        dx, dgamma, dbeta = moe.moe_layernorm_backward(s["dy"], s["x"], s["gamma"], mean, rstd, dres=s.get("dres"))
        return {"y": y, "mean": mean, "rstd": rstd, "dx": dx, "dgamma": dgamma, "dbeta": dbeta}
    dt, wdt = _TYPES[c["dtype"]], _TYPES[c["wdtype"]]
    x, gamma, beta = s["x"].float(), s["gamma"].float(), s["beta"].float()
    mean = x.mean(1)
    xc = x - mean[:, None]
    rstd = 1.0 / torch.sqrt((xc * xc).mean(1) + _EPS)
    xhat = xc * rstd[:, None]
    y = (xhat * gamma + beta).to(dt)
    if not c["train"]:
        return {"y": y}
    dy = s["dy"].float()
    g = dy * gamma
    dx = rstd[:, None] * (g - g.mean(1, keepdim=True) - xhat * (g * xhat).mean(1, keepdim=True))
    if c["dres"]:
        dx = dx + s["dres"].float()
    return {"y": y, "mean": mean, "rstd": rstd, "dx": dx.to(dt), "dgamma": (dy * xhat).sum(0).to(wdt), "dbeta": dy.sum(0).to(wdt)}


def _threshold(p):
    """An element is dropped where its 16-bit uniform number is below this: p in steps of 2^-16."""
    return int(math.floor(p * 65536 + 0.5))


def _keep(T, d, seed, offset, thr, device):
    """Where dropout keeps. Element i = row * d + column takes 16 bits of the Philox 4x32-10 block (Salmon, Moraes, Dror, Shaw: Parallel
    random numbers: as easy as 1, 2, 3) with key `seed` and counter (i / 8, offset): word (i % 8) / 2, its low half first."""
    low = 0xFFFFFFFF
    block = torch.arange((T * d + 7) // 8, device=device, dtype=torch.int64)
    c0, c1 = block & low, block >> 32
    c2, c3 = torch.full_like(block, offset & low), torch.full_like(block, offset >> 32)
    k0, k1 = seed & low, seed >> 32

    def high(a, m):  # the upper 32 bits of a 64-bit product
        return ((a >> 16) * m + (((a & 0xFFFF) * m) >> 16)) >> 16

    for _ in range(10):
        h0, l0 = high(c0, 0xD2511F53), (c0 * 0xD2511F53) & low
        h1, l1 = high(c2, 0xCD9E8D57), (c2 * 0xCD9E8D57) & low
        c0, c1, c2, c3 = h1 ^ c1 ^ k0, l1, h0 ^ c3 ^ k1, l0
        k0, k1 = (k0 + 0x9E3779B9) & low, (k1 + 0xBB67AE85) & low
    words = torch.stack([c0, c1, c2, c3], 1)
    halves = torch.stack([words & 0xFFFF, words >> 16], 2)
    return (halves.reshape(-1)[: T * d] >= thr).reshape(T, d)


def _run_dropout(s):
    c = s["case"]
    if own:
        from top_routing_grouped_02_gb300 import moe

        y = moe.moe_dropout(s["x"], c["p"], s["seed"], s["offset"], residual=s.get("res"))
        if not c["train"]:
            return {"y": y}
        return {"y": y, "dx": moe.moe_dropout_backward(s["dy"], c["p"], s["seed"], s["offset"])}
    dt, thr = _TYPES[c["dtype"]], _threshold(c["p"])
    scale = 65536.0 / (65536 - thr)
    keep = _keep(c["T"], c["d"], s["seed"], s["offset"], thr, s["x"].device)
    y = torch.where(keep, s["x"].float() * scale, 0.0)
    if c["residual"]:
        y = y + s["res"].float()
    if not c["train"]:
        return {"y": y.to(dt)}
    return {"y": y.to(dt), "dx": torch.where(keep, s["dy"].float() * scale, 0.0).to(dt)}


_C0, _C1 = math.sqrt(2.0 / math.pi), 0.044715


def _act(a, act):
    """The activation and its derivative."""
    if act == "silu":
        sg = 1.0 / (1.0 + torch.exp(-a))
        return a * sg, sg * (1.0 + a * (1.0 - sg))
    t = torch.tanh(_C0 * (a + _C1 * a * a * a))
    return 0.5 * a * (1.0 + t), 0.5 * (1.0 + t) + 0.5 * a * (1.0 - t * t) * _C0 * (1.0 + 3.0 * _C1 * a * a)


def _run_ffn(s):
    c = s["case"]
    if own:
        from top_routing_grouped_02_gb300 import moe

        if not c["train"]:
            return {"y": moe.moe_ffn(s["x"], s["w1"], s["w3"], s["w2"], act=c["act"], ws=s["ws"])}
        y, h, a1, a3 = moe.moe_ffn_train(s["x"], s["w1"], s["w3"], s["w2"], act=c["act"], ws=s["ws"])
        dx, dw1, dw3, dw2 = moe.moe_ffn_backward(s["dy"], s["x"], s["w1"], s["w3"], s["w2"], h, a1, a3, act=c["act"], ws=s["ws"])
        return {"y": y, "dx": dx, "dw1": dw1, "dw3": dw3, "dw2": dw2}
    dt = _TYPES[c["dtype"]]
    x, w1, w3, w2 = (s[k].float() for k in ("x", "w1", "w3", "w2"))
    a1, a3 = x @ w1, x @ w3
    f, df = _act(a1, c["act"])
    h = f * a3
    y = (h @ w2).to(dt)
    if not c["train"]:
        return {"y": y}
    dy = s["dy"].float()
    dw2 = (h.T @ dy).to(dt)
    dh = dy @ w2.T
    da1, da3 = dh * a3 * df, dh * f
    dx = (da1 @ w1.T + da3 @ w3.T).to(dt)
    return {"y": y, "dx": dx, "dw1": (x.T @ da1).to(dt), "dw3": (x.T @ da3).to(dt), "dw2": dw2}


# --------------------------------------------------------------------------- what a pass cannot do without


def work(case):
    T, d = case["T"], case["d"]
    e = 4 if case["dtype"] == "fp32" else 2
    if case["op"] == "ffn":
        n, act, wts = case["n"], 2 * T * d * e, 3 * d * case["n"] * e
        if not case["train"]:
            return {"bytes": act + wts, "flops": 6 * T * d * n}
        return {"bytes": 2 * act + 2 * wts, "flops": 18 * T * d * n}
    if case["op"] == "dropout":
        streams = 2 + case["residual"] + 2 * case["train"]
        return {"bytes": streams * T * d * e, "flops": 2 * T * d * (1 + case["train"])}
    w = 4 if case["wdtype"] == "fp32" else 2
    if not case["train"]:
        return {"bytes": 2 * T * d * e + 2 * d * w, "flops": 8 * T * d}
    return {"bytes": (4 + case["dres"]) * T * d * e + 4 * d * w + 8 * T, "flops": 20 * T * d}


# --------------------------------------------------------------------------- the definition in 64 bits


def exact(case, seed):
    s = prepare(case, seed)
    return {"layernorm": _exact_layernorm, "dropout": _exact_dropout, "ffn": _exact_ffn}[case["op"]](case, s)


def _exact_layernorm(case, s):
    # with V the row's variance and h = (x - E x) / sqrt(V + eps), L = <dy, gamma h + beta>; the gradient by
    # the quotient rule: dL/dx = (u - E u) / r - (x - E x) * E[(x - E x) u] / r^3, u = gamma dy, r = sqrt(V + eps)
    x, gamma, beta = s["x"].double(), s["gamma"].double(), s["beta"].double()
    d = case["d"]
    m = torch.einsum("td->t", x) / d
    c = x - m.unsqueeze(1)
    r = (torch.einsum("td,td->t", c, c) / d + _EPS).sqrt()
    y = torch.addcmul(beta, c / r.unsqueeze(1), gamma)
    if not case["train"]:
        return {"y": y}
    dy = s["dy"].double()
    u = dy * gamma
    dx = (u - u.sum(1, keepdim=True) / d) / r.unsqueeze(1) - c * (torch.einsum("td,td->t", c, u) / d / r**3).unsqueeze(1)
    if case["dres"]:
        dx += s["dres"].double()
    return {"y": y, "mean": m, "rstd": r.reciprocal(), "dx": dx, "dgamma": torch.einsum("td,td,t->d", dy, c, 1 / r), "dbeta": torch.einsum("td->d", dy)}


def _exact_dropout(case, s):
    T, d = case["T"], case["d"]
    u64 = np.uint64
    low, half = u64(0xFFFFFFFF), u64(32)
    i = np.arange(-(-T * d // 8), dtype=u64)
    ctr = [i & low, i >> half, np.full_like(i, s["offset"] % 2**32), np.full_like(i, s["offset"] // 2**32)]
    key = np.array([s["seed"] % 2**32, s["seed"] // 2**32], dtype=u64)
    for _ in range(10):
        p, q = ctr[0] * u64(0xD2511F53), ctr[2] * u64(0xCD9E8D57)  # 64-bit products of 32-bit numbers: exact
        ctr = [(q >> half) ^ ctr[1] ^ key[0], q & low, (p >> half) ^ ctr[3] ^ key[1], p & low]
        key = (key + np.array([0x9E3779B9, 0xBB67AE85], dtype=u64)) & low
    bits = np.stack(ctr, 1).astype("<u4").view("<u2").reshape(-1)[: T * d].reshape(T, d)
    drop = math.floor(case["p"] * 65536 + 0.5)
    keep = torch.from_numpy(bits >= drop).to(s["x"].device)
    factor = keep.double() / (1 - drop / 65536)
    out = {"y": s["x"].double() * factor}
    if case["residual"]:
        out["y"] += s["res"].double()
    if case["train"]:
        out["dx"] = s["dy"].double() * factor
    return out


def _exact_ffn(case, s):
    # gelu's tanh form is a * sigmoid(2 u), u = c0 (a + c1 a^3): both activations are a * sigmoid(z(a))
    x, w1, w3, w2 = (s[k].double() for k in ("x", "w1", "w3", "w2"))
    a, b = torch.mm(x, w1), torch.mm(x, w3)
    if case["act"] == "silu":
        z, dz = a, torch.ones_like(a)
    else:
        k = 2 * (2 / math.pi) ** 0.5
        z, dz = k * (a + 0.044715 * a**3), k * (1 + 3 * 0.044715 * a**2)
    g = torch.sigmoid(z)
    f = a * g
    y = torch.mm(f * b, w2)
    if not case["train"]:
        return {"y": y}
    dy = s["dy"].double()
    dh = torch.mm(dy, w2.t())
    u, v = dh * b * (g + f * (1 - g) * dz), dh * f
    return {"y": y, "dx": torch.mm(u, w1.t()).addmm_(v, w3.t()), "dw1": torch.mm(x.t(), u), "dw3": torch.mm(x.t(), v), "dw2": torch.mm((f * b).t(), dy)}
