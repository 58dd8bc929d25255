"""simsd_kvq_append and simsd_kvq_verify at the ends of what their header
allows.  Tolerances as in test_gpu_kvq (kvq_ref.verify's bound); what must
not change is compared bit by bit."""
import math

import pytest
import torch

import kvq_ref as ref
import speculative_decoding_diffusion_gb300 as pkg
from test_gpu_kvq import DT, PAGE, Cache, case, check, cu_of, i32, launch, tables

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("order,B,Hq,hd", [("paired", 4, 4, 128), ("causal", 64, 2, 128), ("nodes", 40, 6, 64), ("causal", 3, 8, 64)])
@pytest.mark.parametrize("size", [2.0 ** 12, 1e8, 1e12, 3e38])
def test_verify_finite_outliers_change_no_row_that_does_not_see_them(dtype, order, B, Hq, hd, size):
    """A token's keys and values times `size` (3e38: as large as that): the same bits in the rows that do not see it,
    and in the others what the definition gives."""
    node = 8 if order == "nodes" else 0
    s = case(61, [50, 0], [B, B], order, dtype, Hq, 2, hd, node)
    clean = launch(s)[0].cpu()
    n = 2 * B if order == "paired" else B
    at = {0: 1, 1: n - 1}                                 # a token of each sequence; head 0 of it, head 1

    def grow(x):
        return (x.sign() * size if size > 1e30 else x * size).to(x.dtype)

    for b, token in at.items():
        for t in (s["kn"], s["vn"]):
            t[b * n + token, b] = grow(t[b * n + token, b])
    out, ws = launch(s)
    assert pkg.read_status(ws) == 0
    if size < 1e30:                                       # (a key of 3e38 leaves fp32 where it is seen)
        check(s, out)
    out = out.cpu()
    for b, token in at.items():
        tau = s["tau"][b * B:(b + 1) * B] if order == "paired" else None
        sees = ref.visible(order, B, tau, node)[:, token]
        rows = slice(b * n, (b + 1) * n)
        mine, other = (slice(h * Hq // 2, (h + 1) * Hq // 2) for h in (b, 1 - b))
        assert 0 < int(sees.sum()) < n
        assert torch.equal(out[rows, mine][~sees], clean[rows, mine][~sees])
        assert torch.equal(out[rows, other], clean[rows, other])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_verify_keys_of_every_size_side_by_side(dtype):
    """New keys from 2^-20 to 2^10 of the usual, all seen: the small ones count with their own scores."""
    s = case(62, [0], [8], "nodes", dtype, 4, 2, 128, 8)
    s["kn"] = (s["kn"].float() * torch.exp2(torch.tensor([-20., -10., -4., 0., 0., 3., 10., -1.]))[:, None, None]).to(DT[dtype])
    out, _ = launch(s)
    check(s, out)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("lo,hi", [(135, 150), (180, 200), (40, 60)])
def test_verify_value_scales_that_no_append_writes(dtype, lo, hi):
    """A stored code stands for c 2^(byte - 127) at every byte, in both kernels."""
    s = case(63, [150, 31], [2, 3], "paired", dtype, 4, 2, 128)
    g = torch.Generator().manual_seed(64)
    s["c"].vs = torch.randint(lo, hi, s["c"].vs.shape, generator=g, dtype=torch.int64).to(torch.uint8)
    s["vn"] = (s["vn"].float() * 2.0 ** ((lo + hi) // 2 - 120)).to(DT[dtype])
    out, ws = launch(s)
    assert pkg.read_status(ws) == 0
    check(s, out)


def test_append_of_a_part_of_a_batch():
    """cu_n of the later sequences of a larger batch: their rows, no complaint about the rows before them."""
    g = torch.Generator().manual_seed(68)
    n, start = [40, 25, 3, 18], [0, 7, 16, 30]
    table, total = tables(g, [(s + m + PAGE - 1) // PAGE for s, m in zip(start, n)])
    c = Cache(g, total, 2, 64)
    v = torch.randn(sum(n), 2, 64, generator=g)
    cu, spec = cu_of(n), dict(base=1e4, rotary_dim=2)
    for first in (1, 2, 3):
        dev = c.cuda()
        ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
        pkg.kvq_append(v.cuda(), v.cuda(), i32(start[first:]), i32(cu[first:]), *dev, i32(table[first:]), ws, pkg.rope_spec(**spec))
        assert pkg.read_status(ws) == 0
        wv, wb = ref.append(v.double(), start[first:], cu[first:], table[first:], c.v, c.vs)
        got = [t.cpu() for t in dev]
        assert torch.equal(got[3], wb) and torch.equal(ref.e4m3_values(got[1]), wv)


def test_calls_without_rows():
    """Empty tensors (which have no memory): nothing is done and nothing refused."""
    g = torch.Generator().manual_seed(69)
    spec = pkg.rope_spec(base=1e4)
    none = torch.empty(0, 2, 64, device="cuda")
    pkg.rope(none, i32([]), spec, none, none, none)
    table, total = tables(g, [1, 1])
    dev = Cache(g, total, 2, 64).cuda()
    before = [t.clone() for t in dev]
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    pkg.kvq_append(none, none, i32([3, 5]), i32([0, 0, 0]), *dev, i32(table), ws, spec)
    assert pkg.read_status(ws) == 0 and all(torch.equal(a, b) for a, b in zip(dev, before))
    assert math.isfinite(float(dev[0].float().sum()))


def test_rope_refuses_an_output_whose_rows_or_heads_share_memory():
    x = torch.randn(5, 4, 64, device="cuda")
    pos, spec = i32(torch.arange(5)), pkg.rope_spec(base=1e4)
    one = torch.zeros(5, 1, 64, device="cuda")
    row = torch.zeros(1, 4, 64, device="cuda")
    near = torch.zeros(4096, device="cuda")
    for out in (row.expand(5, 4, 64), one.expand(5, 4, 64), near.as_strided((5, 4, 64), (256, 32, 1)),
                near.as_strided((5, 4, 64), (128, 64, 1)), near.as_strided((5, 4, 64), (64, 128, 1))):
        with pytest.raises(ValueError):
            pkg.rope(x, pos, spec, out)
        with pytest.raises(ValueError):
            pkg.rope(x, pos, spec, torch.empty_like(x), x, out)
    y, z = torch.empty_like(x), near.as_strided((5, 4, 64), (64, 320, 1))      # heads first
    pkg.rope(row.expand(5, 4, 64), pos, spec, y)                               # an input may
    pkg.rope(x, pos, spec, y)
    pkg.rope(x, pos, spec, z)
    assert torch.equal(y, z)
