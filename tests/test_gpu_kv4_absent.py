"""simsd_kv4_verify with pages that are not there: their keys count as absent,
compared with 64 bits over the keys that are left (bounds as in test_gpu_kv4, and
each product off by 2^-32 of its row's largest)."""
import math

import pytest
import torch

import kv4_absent_ref as absent
import speculative_decoding_diffusion_gb300 as pkg
from test_gpu_kv4 import case, close, i32, verify

pytestmark = pytest.mark.gpu


def without(table, gone, num_pages):
    """The table with the pages gone[b] out of the cache, each in another way."""
    t, ids = table.clone(), [-1, num_pages, -2 ** 31, 2 ** 31 - 1]
    for b, pages in enumerate(gone):
        for i, p in enumerate(pages):
            t[b, p] = ids[(b + i) % 4]
    return t


def check(seed, lens, gone, Bs, order, dtype, G, Hkv, hd, node=0):
    cache, table, cu, q, kn, vn, tau = case(seed, lens, Bs, order, dtype, G, Hkv, hd)
    spec, scale = dict(base=1e4), 1 / math.sqrt(hd)
    out, ws = verify(q.cuda(), cache.cuda(), without(table, gone, cache.shape[0]), kn.cuda(), vn.cuda(), i32(tau), lens, cu, max(Bs),
                     spec, scale, order, node)
    assert pkg.read_status(ws) == 2
    want, off = absent.verify(q, cache, table, kn, vn, tau, lens, cu, spec, scale, order, node, 2.0 ** -11 if dtype == "bf16" else 0.0, gone)
    top = float(vn.abs().max()) + 6 * 2.0                                     # (scales of the cases: up to 2)
    close(out, want, off + (2.0 ** -32 * (max(lens) + 64) * top if dtype == "bf16" else 0.0), dtype)


@pytest.mark.parametrize("hd", [128, 64])
@pytest.mark.parametrize("dtype,B", [("bf16", 2), ("bf16", 4), ("bf16", 8), ("bf16", 16), ("bf16", 32), ("f32", 2), ("f32", 16)])
def test_pages_of_many_blocks(dtype, B, hd):
    """8 to 128 rows; enough units that a long prompt is one CTA's: first, middle and last pages, a whole block, two of a
    block, all of a prompt."""
    long = 9000 if B <= 4 else 2700                                           # (16 blocks of a warp, of a CTA, and more)
    last = (long + 15) // 16 - 1
    lens = [long, 2333, 300, 40, 129] + [0] * 330
    gone = [[0, 7, 8, 100, 101, last] + list(range(112, 120)) + [130, 140, 150, 160], [9, 17, 26, 64, 127, 128, 135, 145], [18],
            [0, 1, 2], [8]] + [[]] * 330
    Bs = [B, max(1, B - 1), B, B, 1] + [1] * 330
    check(B + hd, lens, gone, Bs, "causal", dtype, 4, 2, hd)


@pytest.mark.parametrize("hd", [128, 64])
@pytest.mark.parametrize("dtype,order,B,node", [("bf16", "paired", 1, 0), ("bf16", "paired", 5, 0), ("bf16", "paired", 16, 0),
                                                ("bf16", "nodes", 8, 4), ("bf16", "nodes", 64, 16), ("f32", "paired", 5, 0)])
def test_pages_of_split_keys(dtype, order, B, node, hd):
    """Few sequences: the missing pages are of several splits, one split has none left."""
    lens = [3000, 77, 1025]
    gone = [list(range(0, 24)) + [50, 99, 187], [1, 4], [63, 64]]
    check(B, lens, gone, [B] * 3, order, dtype, 4, 1, hd, node)


@pytest.mark.parametrize("G,B", [(1, 8), (3, 3), (16, 1), (17, 1), (3, 6), (31, 1), (16, 2), (33, 1), (43, 3)])
@pytest.mark.parametrize("hd", [128, 64])
def test_rows_around_the_kernels_borders(G, B, hd):
    """8, 9, 16, 17, 18, 31, 32, 33 and 129 rows of a KV head: every row is written, by whichever kernel takes them."""
    check(G + B, [200, 0, 1300], [[2], [], [0, 80]], [B] * 3, "causal", "bf16", G, 2, hd)
