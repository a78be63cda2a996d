"""Layer norm of rows past 2^30 elements: two arrays of their weight gradients pass 2^31."""
import pytest
import torch

from top_routing_grouped_02_gb300 import moe

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("d", [2 ** 30 + 8, 2 ** 30 + 6, 2 ** 31 - 2])
def test_longest_rows(d):
    # x alternates 1, -1 (every partial sum is a whole number that fp32 holds); dy is 1 at
    # every fourth element. So mean 0, variance 1, xhat = r x, and dx = r (dy - 1/4 - x/4)
    # to within r^2 - 1 = -1e-5 and a few 2^-24 of the sums
    x = torch.ones(1, d, dtype=torch.bfloat16, device="cuda")
    x[0, 1::2] = -1
    dy = torch.zeros_like(x)
    dy[0, ::4] = 1
    y, mean, rstd = moe.moe_layernorm(x, stats=True)
    assert abs(float(mean)) < 1e-6 and abs(float(rstd) - (1 + 1e-5) ** -0.5) < 1e-6
    assert torch.equal(y, x)  # r = 1 - 5e-6 rounds to 1 in bf16
    del y
    dx, dgamma, dbeta = moe.moe_layernorm_backward(dy, x, None, mean, rstd, wdtype=torch.bfloat16)
    assert torch.equal(dbeta, dy[0])
    assert torch.equal(dgamma, dy[0])
    want = (0.5, 0.0, -0.5, 0.0)
    for k in range(4):
        got = dx[0, k::4]
        # bf16's half step of 0.5, and 2e-5 of r and the sums
        assert float((got.float() - want[k]).abs().max()) <= abs(want[k]) * 2.0 ** -8 + 2e-5
