"""More operators of a transformer's feed-forward sub-block with routed experts, as cases to measure.

  dispatch  every token's row copied to its rows among the rows sorted by expert, and the gradient of that: the sum over a
            token's rows, with the residual branch's gradient added in
  combine   the way back: the experts' rows weighted by the router's weights and summed per token, onto the residual stream;
            its gradients for the rows and for the weights
  norm      the norms behind a block and in front of the next one, in one pass over the stream:
              y = scale x + sigmoid(gate) post(b),  u = pre(y),   post, pre: RMS norms with weights
            with a gate for each row or for each element, and its gradients
  linear    a dense projection with its epilogue, Y = act(X W + bias) + residual, and its gradients

`own` chooses between the plain form below (elementary torch operations in 32 bits) and this framework's calls.
"""
import math

import torch

own = False

_TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
_EPS = 1e-6


# --------------------------------------------------------------------------- cases


def _rows(op, T, K, E, d, dtype, train, res=False, drop=0.0, ld=0):
    return {"op": op, "T": T, "K": K, "E": E, "d": d, "dtype": dtype, "train": train, "res": res, "drop": drop, "ld": ld or d}


def _nm(T, d, dtype, wdtype, gate, scale, train, ld=0):
    return {"op": "norm", "T": T, "d": d, "dtype": dtype, "wdtype": wdtype, "gate": gate, "scale": scale, "train": train, "ld": ld or d}


def _li(T, k, n, dtype, bdtype, act, res, train):
    return {"op": "linear", "T": T, "k": k, "n": n, "dtype": dtype, "bdtype": bdtype, "act": act, "res": res, "train": train}


def listed():
    return [
        # sixteen decoding sequences at the DeepSeek-V3-shaped layer: latency
        dict(_rows("dispatch", 16, 8, 256, 7168, "bf16", False), name="dispatch_16_tokens"),
        # a training step of that layer, with the residual branch's gradient added on the way back
        dict(_rows("dispatch", 4096, 8, 256, 7168, "bf16", True, res=True), name="dispatch_train_4096x7168"),
        # one new token at the Mixtral-shaped layer: latency alone
        dict(_rows("combine", 1, 2, 8, 4096, "bf16", False, res=True), name="combine_one_token"),
        # a training step at the SonicMoE-shaped layer in 16-bit floats
        dict(_rows("combine", 16384, 8, 128, 1536, "fp16", True, res=True), name="combine_train_16384x1536"),
        # an odd width in 32 bits, rows in a wider buffer, experts whose capacity was full: a tenth of the slots has no row
        dict(_rows("combine", 1023, 3, 17, 2047, "fp32", True, drop=0.1, ld=2050), name="combine_train_odd_fp32"),
        # one new token behind a block with a gate for the row: latency
        dict(_nm(1, 4096, "bf16", "bf16", "row", 1.0, False), name="norm_one_token"),
        # a training step of the widest layer with a gate for every element
        dict(_nm(8192, 7168, "bf16", "bf16", "full", 1.0, True), name="norm_train_8192x7168"),
        # an odd width in 32 bits with a scaled residual stream: no row but the first starts on a 16-byte boundary
        dict(_nm(1537, 1023, "fp32", "fp32", "row", 0.5, True), name="norm_train_odd_fp32"),
        # one new token through a down projection of the Mixtral-shaped expert's size onto the residual: the weights are streamed
        dict(_li(1, 14336, 4096, "bf16", "bf16", "none", True, False), name="linear_one_token"),
        # a short prompt through a projection of the DeepSeek-V3-shaped layer's sizes, 16-bit floats
        dict(_li(512, 7168, 2048, "fp16", "fp16", "gelu", True, False), name="linear_512_tokens"),
        # a training step with ragged sizes: no dimension is a multiple of a tile
        dict(_li(777, 1000, 2728, "bf16", "fp32", "gelu", True, True), name="linear_train_ragged"),
        # a training step of an up projection of the Mixtral-shaped expert's size: the largest
        dict(_li(4096, 4096, 14336, "bf16", "bf16", "silu", False, True), name="linear_train_4096"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["dispatch", "combine", "norm", "linear"])
    train = rng.random() < 0.6
    if op == "linear":
        # widths in steps of 8, as the call takes them; any number of tokens
        k, n = 8 * _log(rng, 16, 1792), 8 * _log(rng, 16, 1792)
        T = _log(rng, 64, min(8192, 4096 * 4096 * 14336 // (k * n))) if train else _log(rng, 1, 2048)
        dtype = rng.choice(["bf16", "bf16", "fp16"])
        return _li(T, k, n, dtype, rng.choice([dtype, "fp32"]), rng.choice(["none", "silu", "gelu"]), rng.random() < 0.5, train)
    d = _log(rng, 64, 8192)
    if rng.random() < 0.6:
        d = (d + 7) // 8 * 8
    dtype = rng.choice(["bf16", "bf16", "fp16", "fp32"])
    ld = d + rng.choice([0, 0, 0, 8, 3])
    if op == "norm":
        T = _log(rng, 1, min(16384, 8192 * 7168 // d))
        return _nm(T, d, dtype, rng.choice([dtype, "fp32"]), rng.choice(["none", "row", "full"]), rng.choice([1.0, 1.0, 0.5, 2.5]), train, ld)
    K = rng.randint(1, 8)
    E = _log(rng, K, 256)
    T = _log(rng, 1, min(32768, 4096 * 8 * 7168 // (K * d)))
    return _rows(op, T, K, E, d, dtype, train, rng.random() < 0.5, rng.choice([0.0, 0.0, 0.1]), ld)


def _row_map(c, g):
    """[T * K] int32: the row of each token's slot among the rows sorted by expert (stable), -1 where it has none."""
    T, K, E, R = c["T"], c["K"], c["E"], c["T"] * c["K"]
    logits = torch.randn(T, E, generator=g, device="cuda") + torch.randn(E, generator=g, device="cuda")  # some experts are busier
    expert = logits.topk(K, 1).indices.reshape(-1)
    gone = torch.randperm(R, generator=g, device="cuda")[: int(R * c["drop"])]
    expert[gone] = E  # behind all others
    order = torch.sort(expert, stable=True).indices
    row = torch.empty(R, dtype=torch.int64, device="cuda")
    row[order] = torch.arange(R, device="cuda")
    row[gone] = -1
    return row.int()


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    dt = _TYPES[case["dtype"]]

    def normal(*shape, scale=1.0, dtype=dt, shift=None):
        v = torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32).mul_(scale)
        return (v if shift is None else v.add_(shift)).to(dtype)

    s, T = {"case": dict(case)}, case["T"]
    if case["op"] == "linear":
        k, n = case["k"], case["n"]
        s |= {"x": normal(T, k), "w": normal(k, n, scale=k**-0.5), "bias": normal(n, scale=0.5, dtype=_TYPES[case["bdtype"]])}
        if case["res"]:
            s["res"] = normal(T, n, scale=2.0)
        if case["train"]:
            s["dy"] = normal(T, n)
        if own:  # the scratch memory that a user's program keeps between calls
            from top_routing_grouped_02_gb300 import moe

            s["ws"] = moe.linear_workspace(T, k, n, train=case["train"])
        return s
    d, ld = case["d"], case["ld"]
    if case["op"] == "norm":
        # a residual stream: channels with offsets of their own; a block's output of another scale in each row
        wdt = _TYPES[case["wdtype"]]
        shift = normal(ld, dtype=torch.float32) * 0.5
        s["x"] = normal(T, ld, scale=2.0, shift=shift)[:, :d]
        s["b"] = (normal(T, ld, dtype=torch.float32) * normal(T, 1, dtype=torch.float32).mul_(0.5).exp_()).to(dt)[:, :d]
        if case["gate"] == "full":
            s["gate"] = normal(T, ld, scale=1.5)[:, :d]
        elif case["gate"] == "row":
            s["gate"] = normal(T, scale=1.5, dtype=torch.float32)
        s |= {"post": normal(d, scale=0.2, dtype=wdt, shift=1.0), "pre": normal(d, scale=0.2, dtype=wdt, shift=1.0)}
        if case["train"]:
            s |= {"dy": normal(T, ld)[:, :d], "du": normal(T, ld)[:, :d]}
        return s
    K = case["K"]
    s["row"] = _row_map(case, g)
    # a map with slots that have no row leaves the rows behind the last one as they were: here the zeros that the user put there
    spare = case["drop"] > 0
    if case["op"] == "dispatch":
        s["x"] = normal(T, ld)[:, :d]
        if spare:
            s["xg"] = torch.zeros(T * K, d, dtype=dt, device="cuda")
        if case["train"]:
            s["dxg"] = normal(T * K, ld)[:, :d]
            if case["res"]:
                s["res"] = normal(T, ld)[:, :d]
        return s
    w = torch.rand(T, K, generator=g, device="cuda") + 0.05
    s |= {"z": normal(T * K, ld)[:, :d], "w": w / w.sum(1, keepdim=True)}
    if case["res"]:
        s["res"] = normal(T, ld, scale=2.0)[:, :d]
    if case["train"]:
        s["dy"] = normal(T, ld)[:, :d]
        if spare:
            s["dz"] = torch.zeros(T * K, d, dtype=dt, device="cuda")
    return s


# --------------------------------------------------------------------------- one pass


def run(s):
    return {"dispatch": _run_dispatch, "combine": _run_combine, "norm": _run_norm, "linear": _run_linear}[s["case"]["op"]](s)


def _sum_rows(rows, row, T, K, weights):
    """[T, d] fp32: the sum over each token's rows, k ascending."""
    row = row.long().view(T, K)
    out = torch.zeros(T, rows.shape[1], dtype=torch.float32, device=rows.device)
    for k in range(K):
        v = rows[row[:, k].clamp_min(0)].float()
        if weights is not None:
            v = v * weights[:, k, None]
        out += torch.where(row[:, k, None] >= 0, v, 0.0)
    return out


def _run_dispatch(s):
    c = s["case"]
    T, K, d = c["T"], c["K"], c["d"]
    if own:
        from top_routing_grouped_02_gb300 import moe

        out = {"xg": moe.moe_dispatch(s["x"], s["row"], K, xg=s.get("xg"))}
        if c["train"]:
            out["dx"] = moe.moe_dispatch_backward(s["dxg"], s["row"], K, residual=s.get("res"))
        return out
    row = s["row"].long()
    slot = (row >= 0).nonzero()[:, 0]
    xg = torch.zeros(T * K, d, dtype=s["x"].dtype, device=row.device)
    xg[row[slot]] = s["x"][slot // K]
    if not c["train"]:
        return {"xg": xg}
    dx = _sum_rows(s["dxg"], s["row"], T, K, None)
    if c["res"]:
        dx = dx + s["res"].float()
    return {"xg": xg, "dx": dx.to(s["x"].dtype)}


def _run_combine(s):
    c = s["case"]
    T, K, d = c["T"], c["K"], c["d"]
    if own:
        from top_routing_grouped_02_gb300 import moe

        out = {"y": moe.moe_combine_weighted(s["z"], s["row"], s["w"], residual=s.get("res"))}
        if c["train"]:
            out["dz"], out["dw"] = moe.moe_combine_weighted_backward(s["dy"], s["z"], s["row"], s["w"], dz=s.get("dz"))
        return out
    dt = s["z"].dtype
    y = _sum_rows(s["z"], s["row"], T, K, s["w"])
    if c["res"]:
        y = y + s["res"].float()
    if not c["train"]:
        return {"y": y.to(dt)}
    row = s["row"].long()
    slot = (row >= 0).nonzero()[:, 0]
    dy = s["dy"].float()
    dz = torch.zeros(T * K, d, dtype=dt, device=row.device)
    dw = torch.zeros(T * K, dtype=torch.float32, device=row.device)
    g = dy[slot // K]
    dz[row[slot]] = (s["w"].reshape(-1)[slot][:, None] * g).to(dt)
    dw[slot] = (g * s["z"][row[slot]].float()).sum(1)
    return {"y": y.to(dt), "dz": dz, "dw": dw.view(T, K)}


def _run_norm(s):
    c = s["case"]
    if own:
        from top_routing_grouped_02_gb300 import moe

        gate, scale = s.get("gate"), c["scale"]
        if not c["train"]:
            y, u = moe.moe_block_norm(s["x"], s["b"], s["post"], s["pre"], gate=gate, scale=scale, eps=_EPS)
            return {"y": y, "u": u}
        y, u, r_post, r_pre = moe.moe_block_norm(s["x"], s["b"], s["post"], s["pre"], gate=gate, scale=scale, eps=_EPS, stats=True)
        dx, db, dgate, dpost, dpre = moe.moe_block_norm_backward(s["dy"], s["du"], s["x"], s["b"], s["post"], s["pre"], r_post, r_pre, gate=gate, scale=scale)
        out = {"y": y, "u": u, "r_post": r_post, "r_pre": r_pre, "dx": dx, "db": db, "dpost": dpost, "dpre": dpre}
        return out if gate is None else out | {"dgate": dgate}
    dt, wdt = _TYPES[c["dtype"]], _TYPES[c["wdtype"]]
    x, b, post, pre = (s[k].float() for k in ("x", "b", "post", "pre"))
    gate = torch.ones((), device=x.device)
    if c["gate"] != "none":
        gate = 1.0 / (1.0 + torch.exp(-s["gate"].float()))
        if c["gate"] == "row":
            gate = gate[:, None]
    r_post = 1.0 / torch.sqrt((b * b).mean(1, keepdim=True) + _EPS)
    bh = b * r_post
    n = bh * post
    y = c["scale"] * x + gate * n
    r_pre = 1.0 / torch.sqrt((y * y).mean(1, keepdim=True) + _EPS)
    yh = y * r_pre
    u = yh * pre
    out = {"y": y.to(dt), "u": u.to(dt)}
    if not c["train"]:
        return out
    dy, du = s["dy"].float(), s["du"].float()
    e = du * pre
    g = dy + r_pre * (e - yh * (e * yh).mean(1, keepdim=True))  # the whole gradient of y
    f = gate * g * post
    out |= {"r_post": r_post[:, 0], "r_pre": r_pre[:, 0], "dx": (c["scale"] * g).to(dt)}
    out["db"] = (r_post * (f - bh * (f * bh).mean(1, keepdim=True))).to(dt)
    out |= {"dpost": (gate * g * bh).sum(0).to(wdt), "dpre": (du * yh).sum(0).to(wdt)}
    if c["gate"] != "none":
        dgate = g * n * (gate * (1.0 - gate))
        out["dgate"] = dgate.to(dt) if c["gate"] == "full" else dgate.sum(1)
    return out


_C0, _C1 = math.sqrt(2.0 / math.pi), 0.044715


def _act(a, act):
    """The activation and its derivative."""
    if act == "none":
        return a, torch.ones_like(a)
    if act == "silu":
        sg = 1.0 / (1.0 + torch.exp(-a))
        return a * sg, sg * (1.0 + a * (1.0 - sg))
    t = torch.tanh(_C0 * (a + _C1 * a * a * a))
    return 0.5 * a * (1.0 + t), 0.5 * (1.0 + t) + 0.5 * a * (1.0 - t * t) * _C0 * (1.0 + 3.0 * _C1 * a * a)


def _run_linear(s):
    c = s["case"]
    if own:
        from top_routing_grouped_02_gb300 import moe

        act = None if c["act"] == "none" else c["act"]
        if not c["train"]:
            return {"y": moe.moe_linear(s["x"], s["w"], s["bias"], act=act, residual=s.get("res"), ws=s["ws"])}
        y, f = moe.moe_linear_train(s["x"], s["w"], s["bias"], act=act, residual=s.get("res"), ws=s["ws"])
        dx, dw, dbias = moe.moe_linear_backward(s["dy"], s["x"], s["w"], f, bias_dtype=s["bias"].dtype, ws=s["ws"])
        return {"y": y, "dx": dx, "dw": dw, "dbias": dbias}
    dt = _TYPES[c["dtype"]]
    x, w = s["x"].float(), s["w"].float()
    f, df = _act(x @ w + s["bias"].float(), c["act"])
    if c["res"]:
        f = f + s["res"].float()
    if not c["train"]:
        return {"y": f.to(dt)}
    da = s["dy"].float() * df
    return {"y": f.to(dt), "dx": (da @ w.T).to(dt), "dw": (x.T @ da).to(dt), "dbias": da.sum(0).to(s["bias"].dtype)}


# --------------------------------------------------------------------------- what a pass cannot do without


def work(case):
    T = case["T"]
    e = 4 if case["dtype"] == "fp32" else 2
    if case["op"] == "linear":
        k, n = case["k"], case["n"]
        b = n * (4 if case["bdtype"] == "fp32" else 2)
        once = (T * k + k * n + T * n * (1 + case["res"])) * e + b
        if not case["train"]:
            return {"bytes": once, "flops": 2 * T * k * n}
        return {"bytes": once + (T * n + T * k + k * n) * e + b, "flops": 6 * T * k * n}
    d = case["d"]
    if case["op"] == "norm":
        w = 4 if case["wdtype"] == "fp32" else 2
        gate = {"none": 0, "row": 4 * T, "full": T * d * e}[case["gate"]]
        fwd = 4 * T * d * e + gate + 2 * d * w
        if not case["train"]:
            return {"bytes": fwd, "flops": 10 * T * d}
        return {"bytes": fwd + 4 * T * d * e + gate + 2 * d * w + 8 * T, "flops": 40 * T * d}
    R = T * case["K"]
    rows = (R - int(R * case["drop"])) * d * e
    toks = T * d * e
    if case["op"] == "dispatch":
        if not case["train"]:
            return {"bytes": toks + rows + 4 * R, "flops": 0}
        return {"bytes": 2 * (toks + rows) + case["res"] * toks + 4 * R, "flops": R * d}
    fwd = rows + (1 + case["res"]) * toks + 8 * R
    if not case["train"]:
        return {"bytes": fwd, "flops": 2 * R * d}
    return {"bytes": fwd + toks + rows + 4 * R, "flops": 5 * R * d}


# --------------------------------------------------------------------------- the definition in 64 bits


def exact(case, seed):
    s = prepare(case, seed)
    return {"dispatch": _exact_dispatch, "combine": _exact_combine, "norm": _exact_norm, "linear": _exact_linear}[case["op"]](case, s)


def _slots(s, K):
    """Pairs (flat slot, row) of the slots that have a row."""
    slot = torch.nonzero(s["row"] >= 0).squeeze(1)
    return slot, s["row"].index_select(0, slot).long()


def _exact_dispatch(case, s):
    K = case["K"]
    slot, row = _slots(s, K)
    x = s["x"].double()
    out = {"xg": torch.zeros(x.shape[0] * K, x.shape[1], dtype=torch.float64, device=x.device).index_copy_(0, row, x.index_select(0, slot // K))}
    if case["train"]:
        dx = s["res"].double() if case["res"] else torch.zeros_like(x)
        out["dx"] = dx.index_add(0, slot // K, s["dxg"].double().index_select(0, row))
    return out


def _exact_combine(case, s):
    K = case["K"]
    slot, row = _slots(s, K)
    z, w = s["z"].double().index_select(0, row), s["w"].double().flatten().index_select(0, slot)
    base = s["res"].double() if case["res"] else torch.zeros(case["T"], case["d"], dtype=torch.float64, device=z.device)
    out = {"y": base.index_add(0, slot // K, torch.einsum("rd,r->rd", z, w))}
    if case["train"]:
        dy = s["dy"].double().index_select(0, slot // K)
        out["dz"] = torch.zeros(case["T"] * K, case["d"], dtype=torch.float64, device=z.device).index_copy_(0, row, torch.einsum("rd,r->rd", dy, w))
        out["dw"] = torch.zeros(case["T"] * K, dtype=torch.float64, device=z.device).index_copy_(0, slot, torch.einsum("rd,rd->r", dy, z)).view(-1, K)
    return out


def _exact_norm(case, s):
    # the definition, differentiated by torch in 64 bits
    names = [k for k in ("x", "b", "gate", "post", "pre") if k in s]
    v = {k: s[k].double().requires_grad_(case["train"]) for k in names}
    n2 = torch.linalg.vector_norm(v["b"], dim=1, keepdim=True).square() / case["d"]
    r_post = (n2 + _EPS).rsqrt()
    n = v["b"] * r_post * v["post"]
    if case["gate"] != "none":
        gate = torch.sigmoid(v["gate"])
        n = n * (gate if case["gate"] == "full" else gate.unsqueeze(1))
    y = v["x"] * case["scale"] + n
    r_pre = (torch.einsum("td,td->t", y, y) / case["d"] + _EPS).rsqrt()
    u = torch.einsum("td,t,d->td", y, r_pre, v["pre"])
    out = {"y": y.detach(), "u": u.detach()}
    if case["train"]:
        grads = torch.autograd.grad([y, u], [v[k] for k in names], [s["dy"].double(), s["du"].double()])
        out |= {"r_post": r_post.detach().squeeze(1), "r_pre": r_pre.detach()} | {"d" + k: gr for k, gr in zip(names, grads)}
    return out


def _exact_linear(case, s):
    # gelu's tanh form is a * sigmoid(2 u), u = c0 (a + c1 a^3): it and silu are a * sigmoid(z(a))
    x, w = s["x"].double(), s["w"].double()
    a = torch.addmm(s["bias"].double(), x, w)
    if case["act"] == "none":
        f, df = a, None
    else:
        k = 2 * (2 / math.pi) ** 0.5
        z, dz = (a, 1.0) if case["act"] == "silu" else (k * (a + 0.044715 * a**3), k * (1 + 3 * 0.044715 * a**2))
        g = torch.sigmoid(z)
        f = a * g
        df = g + f * (1 - g) * dz
    y = f + s["res"].double() if case["res"] else f
    if not case["train"]:
        return {"y": y}
    da = s["dy"].double() if df is None else s["dy"].double() * df
    return {"y": y, "dx": torch.mm(da, w.t()), "dw": torch.mm(x.t(), da), "dbias": torch.einsum("tn->n", da)}
