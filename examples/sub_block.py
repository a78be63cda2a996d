"""A transformer's feed-forward sub-block on the library's calls, forward and backward:

    u = layernorm(h)
    y = h + dropout(routed_experts(u)) + dropout(shared_expert(u))

The routed experts are the MoE layer (moe_route .. moe_combine and its backward), the
shared expert the dense gated block (moe_ffn_*). Run as a script it takes a few SGD
steps towards a random target and prints the loss; `forward_tokens` is the same
sub-block for decoding, without dropout and saved tensors.

    python examples/sub_block.py [--tokens 1024] [--steps 5]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from top_routing_grouped_02_gb300 import moe  # noqa: E402

EPS = 1e-5


def init(d, E, n, n_shared, seed=0, device="cuda"):
    """Parameters: norm and router in fp32, the experts in bf16."""
    g = torch.Generator(device).manual_seed(seed)

    def normal(*shape, scale, dtype=torch.bfloat16):
        return (torch.randn(*shape, generator=g, device=device) * scale).to(dtype)

    return dict(
        gamma=torch.ones(d, device=device), beta=torch.zeros(d, device=device),
        Wr=normal(d, E, scale=d ** -0.5, dtype=torch.float32),
        W1=normal(E, d, n, scale=d ** -0.5), W3=normal(E, d, n, scale=d ** -0.5),
        W2=normal(E, n, d, scale=n ** -0.5),
        V1=normal(d, n_shared, scale=d ** -0.5), V3=normal(d, n_shared, scale=d ** -0.5),
        V2=normal(n_shared, d, scale=n_shared ** -0.5))


def workspaces(T, p, K):
    """The scratch memory that a program keeps for T tokens."""
    E, d, n = p["W1"].shape
    return dict(moe=moe.workspace(T, d, E, K, n),
                ffn=moe.ffn_workspace(T, d, p["V1"].shape[1], train=True))


def forward(h, p, K, drop, seed, step, ws):
    """(y, saved): one training forward; step numbers the dropout masks."""
    T, d = h.shape
    E = p["W1"].shape[0]
    u, mean, rstd = moe.moe_layernorm(h, p["gamma"], p["beta"], EPS, stats=True)
    logits = torch.empty((T, E), dtype=torch.float32, device=h.device)
    idx, w, counts = moe.moe_route(u, p["Wr"], K, logits=logits)
    g = moe.moe_permute(idx, E, counts=counts, ws=ws["moe"])
    H, A1, A3 = moe.moe_gemm_gate_up_train(u, p["W1"], p["W3"], g["perm_token"], g["offsets"], K,
                                           ws=ws["moe"])
    Z = moe.moe_gemm_down(H, p["W2"], w.view(-1), g["perm_slot"], g["offsets"], T, K, ws=ws["moe"])
    routed = moe.moe_combine(Z, g["row_of_slot"], K)
    shared, S, F1, F3 = moe.moe_ffn_train(u, p["V1"], p["V3"], p["V2"], ws=ws["ffn"])
    y = moe.moe_dropout(routed, drop, seed, 2 * step, residual=h)
    y = moe.moe_dropout(shared, drop, seed, 2 * step + 1, residual=y, y=y)
    return y, dict(h=h, u=u, mean=mean, rstd=rstd, logits=logits, idx=idx, w=w, g=g, H=H, A1=A1,
                   A3=A3, S=S, F1=F1, F3=F3)


def backward(dy, s, p, K, drop, seed, step, ws):
    """(dh, gradients by parameter name) of forward."""
    g, u = s["g"], s["u"]
    drouted = moe.moe_dropout_backward(dy, drop, seed, 2 * step)
    dshared = moe.moe_dropout_backward(dy, drop, seed, 2 * step + 1)
    du_s, dV1, dV3, dV2 = moe.moe_ffn_backward(dshared, u, p["V1"], p["V3"], p["V2"], s["S"], s["F1"],
                                               s["F3"], ws=ws["ffn"])
    w = s["w"].view(-1)
    dA1, dA3, dS = moe.moe_backward_dh(drouted, p["W2"], s["A1"], s["A3"], w, g["perm_token"],
                                       g["perm_slot"], g["offsets"], K, ws=ws["moe"])
    dXg, _ = moe.moe_backward_dx(dA1, dA3, p["W1"], p["W3"], g["offsets"], g["row_of_slot"], K,
                                 ws=ws["moe"])
    dw = moe.moe_backward_dw(u, drouted, s["H"], dA1, dA3, w, g["perm_token"], g["perm_slot"],
                             g["offsets"], K)
    router = moe.moe_backward_router(u, p["Wr"], s["logits"], s["idx"], dS, g["row_of_slot"], dXg,
                                     ws=ws["moe"])
    # the two branches' gradients of u: a residual sum without dropout
    du = moe.moe_dropout(router["dX"], 0.0, 0, residual=du_s, y=du_s)
    dh, dgamma, dbeta = moe.moe_layernorm_backward(du, s["h"], p["gamma"], s["mean"], s["rstd"], dres=dy)
    return dh, dict(gamma=dgamma, beta=dbeta, Wr=router["dWr"], W1=dw["dW1"], W3=dw["dW3"],
                    W2=dw["dW2"], V1=dV1, V3=dV3, V2=dV2)


def forward_tokens(h, p, K, ws):
    """The sub-block for new tokens (inference)."""
    u = moe.moe_layernorm(h, p["gamma"], p["beta"], EPS)
    routed = moe.moe_forward(u, p["Wr"], p["W1"], p["W3"], p["W2"], K, ws=ws["moe"])
    shared = moe.moe_ffn(u, p["V1"], p["V3"], p["V2"], ws=ws["ffn"])
    y = moe.moe_dropout(routed, 0.0, 0, residual=h)
    return moe.moe_dropout(shared, 0.0, 0, residual=y, y=y)


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--tokens", type=int, default=1024)
    ap.add_argument("--steps", type=int, default=5)
    ap.add_argument("--lr", type=float, default=2.0)
    a = ap.parse_args()
    T, d, E, K, n, n_shared, drop, seed = a.tokens, 512, 8, 2, 512, 1024, 0.1, 42
    p = init(d, E, n, n_shared)
    ws = workspaces(T, p, K)
    g = torch.Generator("cuda").manual_seed(1)
    h, target = (torch.randn(T, d, generator=g, device="cuda").bfloat16() for _ in range(2))
    for step in range(a.steps):
        y, saved = forward(h, p, K, drop, seed, step, ws)
        diff = y.float() - target.float()
        _, grads = backward((diff * (2 / T)).bfloat16(), saved, p, K, drop, seed, step, ws)
        print(f"step {step}: loss {float(diff.square().sum(1).mean()):.3f}")
        for name, grad in grads.items():
            p[name] -= (a.lr / d * grad.float()).to(p[name].dtype)
    print("next token:", tuple(forward_tokens(h[:1], p, K, ws).shape))
    for name, w in ws.items():
        status, word = moe.moe_sync_check(w)
        assert status == 0, f"{name}: device error word {word:#x}"


if __name__ == "__main__":
    main()
