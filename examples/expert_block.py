"""A transformer's block of plain experts with biases between two norms, on the library's calls:

    u = rms(h) pre
    routed = sum over a token's K experts e of w_e ((gelu(u A[e] + a[e])) B[e] + b[e])
    h' = h + sigmoid(u g) rms(routed) post,   u' = rms(h') pre'

i.e. the experts are two projections with biases each (moe_linear), their rows come sorted by
expert (moe_route, moe_permute, moe_dispatch), go back weighted (moe_combine_weighted), and one
pass adds them to the stream behind a norm and a gate of the row and makes the next block's
input (moe_block_norm). `forward` and `backward` are a training step of it, for some tens of experts: each
one's projections are launches of their own, over runs of rows that the host reads.

    python examples/expert_block.py [--tokens 1024] [--steps 5]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from top_routing_grouped_02_gb300 import moe  # noqa: E402

EPS = 1e-6


def init(d, E, n, seed=0, device="cuda"):
    """Parameters: norms, router, gate and biases in fp32, the experts' matrices in bf16."""
    g = torch.Generator(device).manual_seed(seed)

    def normal(*shape, scale, dtype=torch.float32):
        return (torch.randn(*shape, generator=g, device=device) * scale).to(dtype)

    return dict(
        pre=torch.ones(d, device=device), post=torch.ones(d, device=device), next=torch.ones(d, device=device),
        Wr=normal(d, E, scale=d ** -0.5), gate=normal(d, scale=d ** -0.5),
        A=normal(E, d, n, scale=d ** -0.5, dtype=torch.bfloat16), a=normal(E, n, scale=0.1),
        B=normal(E, n, d, scale=n ** -0.5, dtype=torch.bfloat16), b=normal(E, d, scale=0.1))


def workspaces(T, p, K):
    """The scratch memory that a program keeps for T tokens."""
    E, d, n = p["A"].shape
    return dict(moe=moe.workspace(T, d, E, K, n), up=moe.linear_workspace(T * K, d, n, train=True),
                down=moe.linear_workspace(T * K, n, d, train=True))


def forward(h, p, K, ws):
    """(h', u', saved)."""
    T, d = h.shape
    E = p["A"].shape[0]
    u, r = moe.moe_rmsnorm(h, p["pre"], EPS, stats=True)
    logits = torch.empty(T, E, device=h.device)
    idx, w, counts = moe.moe_route(u, p["Wr"], K, logits=logits)
    m = moe.moe_permute(idx, E, counts=counts, ws=ws["moe"])
    off = m["offsets"].tolist()  # the experts' runs of rows (a program with fixed runs needs no copy)
    row = m["row_of_slot"]
    xg = moe.moe_dispatch(u, row, K)
    z, experts = torch.empty_like(xg), []
    for e in range(E):
        x = xg[off[e]:off[e + 1]]
        v, F = moe.moe_linear_train(x, p["A"][e], p["a"][e], act="gelu", ws=ws["up"])
        moe.moe_linear(v, p["B"][e], p["b"][e], Y=z[off[e]:off[e + 1]], ws=ws["down"])
        experts.append((v, F))
    y = moe.moe_combine_weighted(z, row, w)
    gate = u.float() @ p["gate"]
    out, nxt, r_post, r_pre = moe.moe_block_norm(h, y, p["post"], p["next"], gate=gate, eps=EPS, stats=True)
    return out, nxt, dict(h=h, u=u, r=r, logits=logits, idx=idx, w=w, off=off, row=row, xg=xg, z=z,
                          experts=experts, y=y, gate=gate, r_post=r_post, r_pre=r_pre)


def backward(dh, du, s, p, K, ws):
    """(the gradient of h, gradients by parameter name), from those of h' and u'."""
    E, off, row = p["A"].shape[0], s["off"], s["row"]
    dres, dy, dgate, dpost, dnext = moe.moe_block_norm_backward(
        dh, du, s["h"], s["y"], p["post"], p["next"], s["r_post"], s["r_pre"], gate=s["gate"])
    dz, dw = moe.moe_combine_weighted_backward(dy, s["z"], row, s["w"])
    dxg = torch.empty_like(s["xg"])
    g = {k: torch.zeros_like(p[k]) for k in ("A", "a", "B", "b")}
    for e in range(E):
        rows = slice(off[e], off[e + 1])
        v, F = s["experts"][e]
        dv, g["B"][e], g["b"][e] = moe.moe_linear_backward(dz[rows], v, p["B"][e], None, bias_dtype=torch.float32,
                                                          ws=ws["down"])
        dxg[rows], g["A"][e], g["a"][e] = moe.moe_linear_backward(dv, s["xg"][rows], p["A"][e], F,
                                                                 bias_dtype=torch.float32, ws=ws["up"])
    # the router's backward takes the weights' gradients by sorted row and adds its share to the experts'
    dS = torch.zeros(row.numel(), device=row.device)
    dS[row.long()] = dw.view(-1)
    router = moe.moe_backward_router(s["u"], p["Wr"], s["logits"], s["idx"], dS, row, dxg, ws=ws["moe"])
    du = moe.moe_dispatch_backward(router["dX"], torch.arange(len(s["u"]), dtype=torch.int32, device=row.device), 1,
                                   residual=(dgate[:, None] * p["gate"]).to(s["u"].dtype))
    dh, dpre = moe.moe_rmsnorm_backward(du, s["h"], p["pre"], s["r"], dres=dres)
    return dh, g | dict(post=dpost, next=dnext, pre=dpre, Wr=router["dWr"], gate=s["u"].float().T @ dgate)


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--tokens", type=int, default=1024)
    ap.add_argument("--steps", type=int, default=5)
    ap.add_argument("--lr", type=float, default=0.5)
    a = ap.parse_args()
    T, d, E, K, n = a.tokens, 512, 8, 2, 1024
    p = init(d, E, n)
    ws = workspaces(T, p, K)
    g = torch.Generator("cuda").manual_seed(1)
    h, target = (torch.randn(T, d, generator=g, device="cuda").bfloat16() for _ in range(2))
    for step in range(a.steps):
        y, _, saved = forward(h, p, K, ws)
        diff = y.float() - target.float()
        _, grads = backward((diff * (2 / T)).bfloat16(), torch.zeros_like(h), saved, p, K, ws)
        print(f"step {step}: loss {float(diff.square().sum(1).mean()):.3f}")
        for name, grad in grads.items():
            p[name] -= (a.lr * grad.float()).to(p[name].dtype)
    for name, w in ws.items():
        status, word = moe.moe_sync_check(w)
        assert status == 0, f"{name}: device error word {word:#x}"


if __name__ == "__main__":
    main()
