"""The layer's combine of weighted rows and the sum of rows without weights are one formula: the same bits."""
import pytest
import torch

from block_common import matrix
from rows_common import slot_map
from top_routing_grouped_02_gb300 import moe

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T,K,d", [(1, 1, 8), (3, 8, 7168), (257, 2, 4096), (1000, 3, 136), (500, 5, 1536)])
def test_same_bits(T, K, d):
    gen = torch.Generator().manual_seed(T + d)
    row = slot_map(T, K, max(K, 4), 0.0, gen)[0].cuda()
    row[torch.randperm(T * K, generator=gen)[: T * K // 7].cuda()] = T * K  # no row
    z = matrix(T * K, d, torch.bfloat16, gen)
    assert torch.equal(moe.moe_combine(z, row, K), moe.moe_dispatch_backward(z, row, K))
