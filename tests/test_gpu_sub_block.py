"""The sub-block of examples/sub_block.py (norm, routed experts, shared expert, residual
dropout) against 64-bit autograd of its definition, with the kernels' top-K choice."""
import importlib.util
import os

import pytest
import torch

from block_common import dropout_scale, keep_mask
from top_routing_grouped_02_gb300 import moe

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
spec = importlib.util.spec_from_file_location("sub_block", os.path.join(ROOT, "examples", "sub_block.py"))
sub_block = importlib.util.module_from_spec(spec)
spec.loader.exec_module(sub_block)

T, d, E, K, n, NS, P, SEED, STEP = 200, 256, 8, 2, 256, 328, 0.25, 99, 3
U = 2.0 ** -8  # half a step of bf16


def plain(h, p, idx, drop):
    """y in 64 bits, differentiable in h and the parameters (all double)."""
    f = torch.nn.functional
    u = f.layer_norm(h, (d,), p["gamma"], p["beta"], sub_block.EPS)
    probs = torch.softmax(u @ p["Wr"], 1).gather(1, idx)
    w = probs / probs.sum(1, keepdim=True)
    routed = torch.zeros_like(h)
    for e in range(E):
        mine = ((idx == e) * w).sum(1, keepdim=True)
        routed = routed + mine * ((f.silu(u @ p["W1"][e]) * (u @ p["W3"][e])) @ p["W2"][e])
    shared = (f.silu(u @ p["V1"]) * (u @ p["V3"])) @ p["V2"]
    if not drop:
        return h + routed + shared
    m = [keep_mask(T * d, P, SEED, 2 * STEP + i).view(T, d).to(h.device) * dropout_scale(P) for i in (0, 1)]
    return h + routed * m[0] + shared * m[1]


def rel(a, b):
    return float((a.double() - b).norm() / b.norm())


def test_training_step():
    p = sub_block.init(d, E, n, NS, seed=5)
    g = torch.Generator("cuda").manual_seed(6)
    p["gamma"] += 0.2 * torch.randn(d, generator=g, device="cuda")
    p["beta"] += 0.2 * torch.randn(d, generator=g, device="cuda")
    h, dy = (torch.randn(T, d, generator=g, device="cuda").bfloat16() for _ in range(2))
    ws = sub_block.workspaces(T, p, K)
    y, saved = sub_block.forward(h, p, K, P, SEED, STEP, ws)
    dh, grads = sub_block.backward(dy, saved, p, K, P, SEED, STEP, ws)
    for w in ws.values():
        assert moe.moe_sync_check(w) == (0, 0)
    leaves = {k: v.double().requires_grad_() for k, v in p.items()}
    hd = h.double().requires_grad_()
    want = plain(hd, leaves, saved["idx"].long(), True)
    want.backward(dy.double())
    # roundings to 16 bits in a row (u each at most): y: u, H, Z, combine, two sums = 6;
    # gradients: those of u and H and the branch gradient, dA, the products' own, the
    # sums of branches: 8
    assert rel(y, want.detach()) <= 6 * U
    assert rel(dh, hd.grad) <= 8 * U
    for name, grad in grads.items():
        assert rel(grad, leaves[name].grad) <= 8 * U, name


def test_tokens():
    p = sub_block.init(d, E, n, NS, seed=7)
    h = torch.randn(3, d, generator=torch.Generator("cuda").manual_seed(8), device="cuda").bfloat16()
    ws = sub_block.workspaces(3, p, K)
    y = sub_block.forward_tokens(h, p, K, ws)
    u = moe.moe_layernorm(h, p["gamma"], p["beta"], sub_block.EPS)
    idx, _, _ = moe.moe_route(u, p["Wr"], K)
    want = plain(h.double(), {k: v.double() for k, v in p.items()}, idx.long(), False)
    assert rel(y, want) <= 6 * U
