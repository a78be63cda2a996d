"""The forms of the block norms' forward: how many elements of a row that starts anywhere a thread takes."""
import re

import pytest
import torch

from launches import kernels
from top_routing_grouped_02_gb300 import moe

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


@pytest.mark.parametrize("d,block,gate,elements", [
    # inputs that start elsewhere than outputs: 16 behind a block, as long as two rows have room
    (2048, True, "row", 16), (4096, True, None, 16), (4096, True, "row", 16), (6144, True, "full", 16), (7160, True, "row", 16),
    (7168, True, "row", 32), (8192, True, "full", 32), (4096, False, None, 32), (2000, False, None, 16)])
def test_elements_of_rows_that_start_elsewhere(d, block, gate, elements):
    T, side = 700, torch.cuda.Stream()
    x, b, z = (torch.zeros(T, d + 3, dtype=BF, device="cuda")[:, :d] for _ in range(3))
    gate = {None: None, "row": torch.zeros(T, device="cuda"), "full": z}[gate]
    call = (lambda: moe.moe_block_norm(x, b, gate=gate, stream=side)) if block else (lambda: moe.moe_rmsnorm(x, stream=side))
    side.wait_stream(torch.cuda.current_stream())
    call()
    (name, _, _), = kernels(call, side)
    vector, vectors, _, places = map(int, re.search(r"forward_ring_kernel.*?Li(\d+)ELi(\d+)ELi(\d+)ELi(\d+)E", name).groups())
    assert places == 2 and vector * vectors == elements, name
