"""simsd_page_map at the ends of its ranges."""
import pytest
import torch

import speculative_decoding_diffusion_gb300 as pkg
from test_gpu_page_map import i32

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("cu,total", [([0, 64, 32, 40], 64), ([0, 40, -5, 8, 20], 40), ([0, 64, 0, 8], 64), ([5, 9, 70, 9, 12], 30),
                                      ([3, 2, 1], 8)])
def test_a_range_that_falls_takes_no_other_sequence_with_it(cu, total):
    """Every sequence whose own range is valid is served and has all its slots (of two that claim a token the later one);
    the others are left as they were."""
    batch, width = len(cu) - 1, 6
    cap = batch * width
    held, served, queue = i32([0] * batch), i32([7] * batch), i32([0, cap])
    ring, table = i32(list(range(cap))), i32([[0] * width] * batch)
    slots = torch.full((total,), -7, dtype=torch.int64, device="cuda")
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    lens = [3 * b for b in range(batch)]
    pkg.page_map(i32(lens), i32(cu), held, queue, ring, table, held, queue, served, slots, ws, total)
    assert pkg.read_status(ws) == 2
    want, page = [-7] * total, 0
    for b in range(batch):
        ok = 0 <= cu[b] <= cu[b + 1] <= total
        n = cu[b + 1] - cu[b] if ok else 0
        pages = (lens[b] + n + 15) // 16 if ok else 0
        assert served[b].item() == int(ok) and held[b].item() == pages
        assert table[b, :pages].tolist() == list(range(page, page + pages))
        for i in range(n):
            want[cu[b] + i] = 16 * (page + (lens[b] + i) // 16) + (lens[b] + i) % 16
        page += pages
    assert slots.tolist() == want and queue.tolist() == [page, cap - page]


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
