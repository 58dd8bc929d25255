"""simsd_kvq_append and simsd_kvq_verify at the ends of what their header
allows.  Tolerances as in test_gpu_kvq (kvq_ref.verify's bound); what must
not change is compared bit by bit."""
import math
import os
import subprocess
import sys

import pytest
import torch

import kvq_ref as ref
import speculative_decoding_diffusion_gb300 as pkg
from test_gpu_kvq import DT, PAGE, Cache, case, check, check_keys, cu_of, i32, launch, tables

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


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("lens,width", [([3000], 1024), ([900, 17, 0], 2048), ([4000, 300] * 4, 640)])
def test_verify_tables_wider_than_the_prompts(dtype, lens, width):
    """A table that leaves room to grow: pieces sized for the table, most of them without keys; ids behind a row's end
    are not read."""
    s = case(65, lens, [2] * len(lens), "paired", dtype, 4, 1, 64)
    tight, _ = launch(s)
    check(s, tight)
    t = torch.full((len(lens), width), 2 ** 30, dtype=s["table"].dtype)
    t[:, :s["table"].shape[1]] = s["table"]
    s["table"] = t
    out, ws = launch(s)
    assert ws.numel() > 256 and pkg.read_status(ws) == 0
    check(s, out)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_attention_factor(dtype):
    """attn_factor on both sides of the scores and in the cache's keys."""
    spec = dict(base=1e4, rotary_dim=64, scaling="linear", factor=2.0, attn_factor=1.25)
    s = case(66, [70, 5], [3, 2], "causal", dtype, 4, 2, 128, spec=spec)
    out, _ = launch(s)
    check(s, out)
    g = torch.Generator().manual_seed(67)
    table, total = tables(g, [3])
    c = Cache(g, total, 2, 128)
    dev = c.cuda()
    k = torch.randn(40, 2, 128, generator=g).to(DT[dtype])
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    pkg.kvq_append(k.cuda(), k.cuda(), i32([0]), i32([0, 40]), *dev, i32(table), ws, pkg.rope_spec(**spec))
    wk, wkb = ref.append(ref.rope(k, torch.arange(40), spec), [0], cu_of([40]), table, c.k, c.ks)
    got = [t.cpu() for t in dev]
    check_keys(got[0], got[2], None, None, wk, wkb)
    y = torch.empty_like(k, device="cuda")
    for inverse in (False, True):
        pkg.rope(k.cuda(), i32(torch.arange(40)), pkg.rope_spec(**spec), y, inverse=inverse)
        want = ref.rope(k, torch.arange(40), spec, inverse)
        size = 1.25 * 2 * k.double().abs().amax(-1, keepdim=True)
        off = 1.5e-6 * size + torch.finfo(DT[dtype]).eps / 2 * want.abs()
        assert ((y.cpu().double() - want).abs() <= off).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_verify_leaves_the_rows_behind_the_last_sequence(dtype):
    """q, k_new, v_new and out longer than the batch needs, with NaN behind it."""
    s = case(70, [40, 3000], [3, 2], "paired", dtype, 4, 1, 64)
    want, _ = launch(s)
    more = {k: torch.cat([s[k], torch.full((7, *s[k].shape[1:]), math.nan, dtype=s[k].dtype)]) for k in ("q", "kn", "vn")}
    out = torch.full(more["q"].shape, 5.0, dtype=DT[dtype], device="cuda")
    out, ws = launch(dict(s, **more), out=out)
    assert pkg.read_status(ws) == 0
    assert torch.equal(out[:10], want) and (out[10:] == 5).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_verify_rows_with_odd_queries_keep_to_themselves(dtype):
    """A NaN or an infinity in a query row: that row and head alone."""
    s = case(71, [60, 20], [5, 5], "causal", dtype, 8, 2, 128)
    clean = launch(s)[0].cpu()
    s["q"][2, 3, 100], s["q"][7, 0, 1] = math.nan, math.inf
    out = launch(s)[0].cpu()
    bad = torch.zeros(10, 8, dtype=torch.bool)
    bad[2, 3] = bad[7, 0] = True
    assert torch.isnan(out[2, 3]).all() and not torch.isfinite(out[7, 0]).any()
    assert torch.equal(out[~bad], clean[~bad])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_verify_sequences_that_share_their_first_pages(dtype):
    """The same page in several rows of the table, and twice in one."""
    s = case(72, [90, 100, 70], [2, 1, 3], "causal", dtype, 4, 2, 64)
    s["table"][1, :4] = s["table"][0, :4]
    s["table"][2, 1:3] = s["table"][2, 0]
    out, ws = launch(s)
    assert pkg.read_status(ws) == 0
    check(s, out)


FIRST = """
import sys
sys.path[:0] = %r
import torch
import speculative_decoding_diffusion_gb300 as pkg
from test_gpu_kvq import case, i32, launch

s = case(73, [300] * 30, [2] * 30, "causal", "bf16", 8, 8, 64)
dev = [t.cuda() for t in (s["q"], *s["c"].cuda(), s["kn"], s["vn"])]
q, cache, kn, vn = dev[0], dev[1:5], dev[5], dev[6]
before = [t.clone() for t in cache]
table, lens, cu, spec = i32(s["table"]), i32(s["lens"]), i32(s["cu"]), pkg.rope_spec(**s["spec"])
start, pos = i32([16] * 30), i32(list(range(60)))
held, queue, ring, served = i32([19] * 30), i32([0, 0]), i32([0] * 600), i32([0] * 30)
slots = torch.zeros(60, dtype=torch.int64, device="cuda")
out, y = torch.zeros_like(q), torch.zeros_like(q)
ws = torch.zeros(1 << 24, dtype=torch.uint8, device="cuda")
wsa, wsm = (torch.zeros(256, dtype=torch.uint8, device="cuda") for _ in range(2))

def calls():
    pkg.rope(q, pos, spec, y)
    pkg.page_map(i32_lens, cu, held, queue, ring, table, held, queue, served, slots, wsm, 60)
    pkg.kvq_append(kn, vn, start, cu, *cache, table, wsa, spec)
    pkg.kvq_verify(q, *cache, table, kn, vn, None, lens, cu, out, ws, 60, 2, spec, s["scale"], order=pkg.SIMSD_ORDER_CAUSAL)

i32_lens = lens.clone()
graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
torch.cuda.synchronize()
with torch.cuda.graph(graph, stream=side):
    calls()
graph.replay()
torch.cuda.synchronize()
first = [t.clone() for t in (out, y, slots, served, *cache)]
for t, old in zip(cache, before):
    t.copy_(old)
calls()
torch.cuda.synchronize()
assert all(torch.equal(a, b) for a, b in zip(first, (out, y, slots, served, *cache)))
assert not (pkg.read_status(ws) | pkg.read_status(wsa) | pkg.read_status(wsm))
print("same")
"""


def test_a_process_whose_first_calls_are_captured():
    """Every call of the loop inside a graph before any outside: what eager calls give."""
    here = os.path.dirname(os.path.abspath(__file__))
    r = subprocess.run([sys.executable, "-c", FIRST % ([here, os.path.dirname(here)],)], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.strip().endswith("same"), r.stdout + r.stderr
