"""The block of examples/expert_block.py (norms, dispatch, experts of two projections, weighted
combine, gate and residual) against 64-bit autograd of its definition, with the kernels' top-K
choice."""
import importlib.util
import os
import subprocess
import sys

import pytest
import torch

from top_routing_grouped_02_gb300 import moe

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
PATH = os.path.join(ROOT, "examples", "expert_block.py")
spec = importlib.util.spec_from_file_location("expert_block", PATH)
block = importlib.util.module_from_spec(spec)
spec.loader.exec_module(block)

T, d, E, K, n = 200, 256, 8, 3, 328
U = 2.0 ** -8  # half a step of bf16


def rms(x):
    return x / torch.sqrt((x * x).mean(1, keepdim=True) + block.EPS)


def plain(h, p, idx):
    """(h', u') in 64 bits, differentiable in h and the parameters (all double)."""
    u = rms(h) * p["pre"]
    probs = torch.softmax(u @ p["Wr"], 1).gather(1, idx)
    w = probs / probs.sum(1, keepdim=True)
    routed = torch.zeros_like(h)
    for e in range(E):
        mine = ((idx == e) * w).sum(1, keepdim=True)
        v = torch.nn.functional.gelu(u @ p["A"][e] + p["a"][e], approximate="tanh")
        routed = routed + mine * (v @ p["B"][e] + p["b"][e])
    y = h + torch.sigmoid(u @ p["gate"])[:, None] * rms(routed) * p["post"]
    return y, rms(y) * p["next"]


def rel(a, b):
    return float((a.double() - b).norm() / b.norm())


def test_training_step():
    p = block.init(d, E, n, seed=5)
    g = torch.Generator("cuda").manual_seed(6)
    for k in ("pre", "post", "next"):
        p[k] += 0.2 * torch.randn(d, generator=g, device="cuda")
    h, dy, du = (torch.randn(T, d, generator=g, device="cuda").bfloat16() for _ in range(3))
    ws = block.workspaces(T, p, K)
    y, u, saved = block.forward(h, p, K, ws)
    dh, grads = block.backward(dy, du, saved, p, K, ws)
    for w in ws.values():
        assert moe.moe_sync_check(w) == (0, 0)
    leaves = {k: v.double().requires_grad_() for k, v in p.items()}
    hd = h.double().requires_grad_()
    want_y, want_u = plain(hd, leaves, saved["idx"].long())
    (want_y * dy.double()).sum().add((want_u * du.double()).sum()).backward()
    # roundings to 16 bits in a row (U each at most, in the 2-norm): u, the hidden rows, z, the
    # combined rows, the output: 5, through a norm whose gradient has a norm of about one
    assert rel(y, want_y.detach()) <= 5 * U and rel(u, want_u.detach()) <= 5 * U
    # those of the forward that the gradients' factors carry (4), then db, dz, dA twice, the
    # experts' row gradients, their sum, the sum of branches, the result's: 8
    assert rel(dh, hd.grad) <= 12 * U
    assert set(grads) == set(p)
    for name, grad in grads.items():
        assert rel(grad, leaves[name].grad) <= 12 * U, name


def test_script_runs():
    out = subprocess.run([sys.executable, PATH, "--tokens", "96", "--steps", "2"], capture_output=True, text=True, timeout=300)
    assert out.returncode == 0, out.stdout + out.stderr
    assert out.stdout.count("loss") == 2
