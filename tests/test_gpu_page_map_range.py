"""simsd_page_map at the ends of its ranges."""
import pytest
import torch

import speculative_decoding_diffusion_gb300 as pkg
from test_gpu_page_map import i32

pytestmark = pytest.mark.gpu


def test_as_many_tokens_as_the_count_holds():
    """2^31 - 1 new tokens: a count of tokens that a step of the grid passes."""
    n, pages = 2 ** 31 - 1, 2 ** 27
    ring = torch.arange(pages - 1, -1, -1, dtype=torch.int32, device="cuda")
    table = torch.zeros(1, pages, dtype=torch.int32, device="cuda")
    held, queue, served = i32([0]), i32([0, pages]), i32([7])
    slots = torch.full((n,), -7, dtype=torch.int64, device="cuda")
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    pkg.page_map(i32([0]), i32([0, n]), held, queue, ring, table, held, queue, served, slots, ws, n)
    assert pkg.read_status(ws) == 0
    assert served.item() == 1 and held.item() == pages and queue.tolist() == [0, 0]
    assert torch.equal(table[0], ring)
    for a in range(0, n, 2 ** 27):
        t = torch.arange(a, min(n, a + 2 ** 27), device="cuda")
        assert torch.equal(slots[a:a + 2 ** 27], (pages - 1 - t // 16) * 16 + t % 16)
