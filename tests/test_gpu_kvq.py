"""simsd_kvq_append and simsd_kvq_verify against their 64-bit forms.

Append.  A stored value is the e4m3 code nearest to x 2^-E.  The kernel's x
is fp32 (a rotation's error: 1.5e-6 (|x1| + |x2|), see test_gpu_rope), so its
code may be the neighbouring one only where the exact value lies that close to
the middle between two codes; the scale may differ only where the exact
maximum lies that close to 448 2^E.  Unrotated values (v) must be equal.

Verify.  kvq_ref.verify gives each output element's bound: scores off by the
query elements' rounding (bf16: two e4m3 parts, 2^-8 of an element, and for
the new tokens' keys as well, so 2 * 2^-8; fp32: none), by
fp32 sums (hd + 16) 2^-24 of the absolute products and 2^-20 |s| for
exponentials; weights off by 2^-11 (f16, for bf16 data) before the product
with the values; then the output's own rounding, half a step."""
import math

import pytest
import torch

import kvq_ref as ref
import speculative_decoding_diffusion_gb300 as pkg

pytestmark = pytest.mark.gpu
PAGE = 16
DT = {"f32": torch.float32, "bf16": torch.bfloat16}


def i32(x):
    return torch.as_tensor(x, dtype=torch.int32).cuda()


def cu_of(n):
    return torch.cat([torch.zeros(1, dtype=torch.int64), torch.as_tensor(n, dtype=torch.int64).cumsum(0)])


def tables(gen, pages, spare=3):
    """Block table with shuffled page ids; entries past a row's end hold an id out of range."""
    pages = torch.as_tensor(pages, dtype=torch.int64)
    total = int(pages.sum()) + spare
    ids = torch.randperm(total, generator=gen)
    t = torch.full((len(pages), max(1, int(pages.max()))), 2 ** 30, dtype=torch.int64)
    at = 0
    for b, n in enumerate(pages.tolist()):
        t[b, :n] = ids[at:at + n]
        at += n
    return t, total


class Cache:
    """Random codes (NaN codes in unused slots stay possible) and scale bytes."""

    def __init__(self, gen, pages, heads, hd, lo=118, hi=124):
        def codes():
            c = torch.randint(0, 256, (pages, heads, PAGE, hd), generator=gen, dtype=torch.int64).to(torch.uint8)
            return torch.where((c & 0x7f) == 0x7f, c & 0xfe, c)
        self.k, self.v = codes(), codes()
        self.ks, self.vs = (torch.randint(lo, hi, (pages, heads), generator=gen, dtype=torch.int64).to(torch.uint8)
                            for _ in range(2))

    def cuda(self):
        return [t.cuda() for t in (self.k, self.v, self.ks, self.vs)]


def put(k, v, start, n, table, dev, spec, take=None, ws=None):
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda") if ws is None else ws
    pkg.kvq_append(k, v, i32(start), i32(cu_of(n)), *dev, i32(table), ws, pkg.rope_spec(**spec),
                   take=None if take is None else i32(take))
    return ws


def check_keys(got_codes, got_bytes, x, size, want_val, want_byte):
    """Codes and scales of rotated keys: equal, or neighbours where the exact value says so."""
    got_val = ref.e4m3_values(got_codes)
    same = (got_val == want_val).all(-1).all(-1) & (got_bytes == want_byte)
    assert (got_bytes == want_byte).float().mean() > 0.99
    off = (got_val * torch.exp2(got_bytes.double() - 127)[..., None, None] -
           want_val * torch.exp2(want_byte.double() - 127)[..., None, None]).abs()
    # a neighbour is at most one step, 2^-3 of the value (or a subnormal step) away, and rare
    step = torch.maximum(want_val.abs() * 2.0 ** -3, torch.tensor(2.0 ** -9, dtype=torch.float64))
    step = step * torch.exp2(torch.maximum(got_bytes, want_byte).double() - 127)[..., None, None]
    assert (off <= step).all()
    assert (off > 0).float().mean() < 1e-3
    return same


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("hd,H", [(128, 2), (64, 9)])
@pytest.mark.parametrize("spec", [dict(base=1e4), dict(base=1e4, interleaved=True, rotary_dim=32),
                                  dict(base=1e6, rotary_dim=48, scaling="linear", factor=2.0),
                                  dict(base=1e6, rotary_dim=50)])
def test_append_matches_definition(dtype, hd, H, spec):
    g = torch.Generator().manual_seed(hd + H)
    start = [0, 5, 16, 31, 100, 7, 0, 15]
    n = [33, 1, 16, 2, 47, 0, 1, 17]
    table, total = tables(g, [(s + m + PAGE - 1) // PAGE for s, m in zip(start, n)])
    c = Cache(g, total, H, hd)
    N = sum(n)
    k = (torch.randn(N, H, hd, generator=g) * torch.exp2(torch.randint(-3, 4, (N, H, 1), generator=g).float())).to(DT[dtype])
    v = (torch.randn(N, H, hd, generator=g) * 3).to(DT[dtype])
    dev = c.cuda()
    ws = put(k.cuda(), v.cuda(), start, n, table, dev, spec)
    assert pkg.read_status(ws) == 0
    cu = cu_of(n)
    pos = torch.cat([torch.arange(s, s + m) for s, m in zip(start, n)])
    xk = ref.rope(k, pos, spec)
    wk, wkb = ref.append(xk, start, cu, table, c.k, c.ks)
    wv, wvb = ref.append(v.double(), start, cu, table, c.v, c.vs)
    got = [t.cpu() for t in dev]
    assert torch.equal(got[3], wvb) and torch.equal(ref.e4m3_values(got[1]), wv)
    check_keys(got[0], got[2], None, None, wk, wkb)
    # the same call again finds the same state
    dev2 = [t.clone() for t in dev]
    put(k.cuda(), v.cuda(), start, n, table, dev2, spec)
    assert all(torch.equal(a, b) for a, b in zip(dev, dev2))


def test_append_scale_borders_zero_and_growth():
    """Maxima at and around 448 2^e, all zeros, the ends of the range; growth
    moves older codes, a smaller newcomer keeps the scale."""
    hd, spec = 64, dict(base=1e4, rotary_dim=2)         # elements 2.. pass unrotated
    tops = [448.0, 449.0, 447.0, 7.0, 7.03125, 0.0, 2.0 ** -60, 57344.0, 60000.0, 3e38, 1e-38, 224.0]
    n = [3] * len(tops)
    table, total = tables(torch.Generator().manual_seed(1), [1] * len(tops))
    c = Cache(torch.Generator().manual_seed(2), total, 1, hd)
    v = torch.zeros(3 * len(tops), 1, hd)
    for i, t in enumerate(tops):
        v[3 * i, 0, 5], v[3 * i + 1, 0, 6], v[3 * i + 2, 0, 7] = t, -t / 3, t * 2.0 ** -12
    k = v.clone()
    k[:, :, :2] = 0
    dev = c.cuda()
    put(k.cuda(), v.cuda(), [0] * len(n), n, table, dev, spec)
    wv, wb = ref.append(v.double(), [0] * len(n), cu_of(n), table, c.v, c.vs)
    wk, wkb = ref.append(k.double(), [0] * len(n), cu_of(n), table, c.k, c.ks)
    got = [t.cpu() for t in dev]
    assert torch.equal(got[3], wb) and torch.equal(ref.e4m3_values(got[1]), wv)
    assert torch.equal(got[2], wkb) and torch.equal(ref.e4m3_values(got[0]), wk)
    # second append behind the first: ten times larger, then a thousand times smaller
    for f in (10.0, 1e-3):
        before = [t.cpu() for t in dev]
        at = [3 if f == 10.0 else 6] * len(n)
        put((k * f).cuda(), (v * f).cuda(), at, n, table, dev, spec)
        wv, wb = ref.append((v * f).double(), at, cu_of(n), table, before[1], before[3])
        got = [t.cpu() for t in dev]
        assert torch.equal(got[3], wb) and torch.equal(ref.e4m3_values(got[1]), wv)


def test_append_nan_and_infinity_mark_the_page():
    hd, g = 64, torch.Generator().manual_seed(5)
    table, total = tables(g, [2, 2])
    c = Cache(g, total, 2, hd)
    dev = c.cuda()
    k, v = torch.randn(40, 2, hd, generator=g), torch.randn(40, 2, hd, generator=g)
    k[3, 0, 63], v[25, 1, 0] = math.nan, -math.inf
    put(k.cuda(), v.cuda(), [0, 0], [20, 20], table, dev, dict(base=1e4))
    ks, vs = dev[2].cpu(), dev[3].cpu()
    assert ks[table[0, 0], 0] == 255 and (ks == 255).sum() == 1
    assert vs[table[1, 0], 1] == 255 and (vs == 255).sum() == 1
    # behind it the mark stays; from the page's first slot it goes
    put(k[4:8].cuda(), v[4:8].cuda(), [4], [4], table[:1], dev, dict(base=1e4))
    assert dev[2].cpu()[table[0, 0], 0] == 255
    put(k[4:8].cuda(), v[4:8].cuda(), [0], [4], table[:1], dev, dict(base=1e4))
    assert dev[2].cpu()[table[0, 0], 0] != 255


def test_append_take_strides_and_untouched_slots():
    """Fused rows, the first take[b] of each sequence's rows, and every slot and page beside them as it was."""
    g = torch.Generator().manual_seed(6)
    H, hd, n, take, start = 3, 128, [8, 8, 8, 8], [4, 0, 8, 1], [14, 3, 16, 0]
    table, total = tables(g, [(s + m + PAGE - 1) // PAGE for s, m in zip(start, n)])
    c = Cache(g, total, H, hd)
    dev = c.cuda()
    rows = torch.randn(sum(n), 2 + 2 * H, hd, generator=g).to(torch.bfloat16)
    d = rows.cuda()
    put(d[:, 2:2 + H], d[:, 2 + H:], start, n, table, dev, dict(base=1e4), take)
    pos = torch.cat([torch.arange(s, s + m) for s, m in zip(start, n)])
    wv, wb = ref.append(rows[:, 2 + H:].double(), start, cu_of(n), table, c.v, c.vs, take)
    wk, wkb = ref.append(ref.rope(rows[:, 2:2 + H], pos, dict(base=1e4)), start, cu_of(n), table, c.k, c.ks, take)
    got = [t.cpu() for t in dev]
    assert torch.equal(got[3], wb) and torch.equal(ref.e4m3_values(got[1]), wv)
    check_keys(got[0], got[2], None, None, wk, wkb)


def test_append_many_sequences_and_bad_arrays():
    g = torch.Generator().manual_seed(7)
    n = [1 + i % 3 for i in range(700)]
    start = [(i * 5) % 40 for i in range(700)]
    table, total = tables(g, [(s + m + PAGE - 1) // PAGE for s, m in zip(start, n)])
    c = Cache(g, total, 1, 64)
    v = torch.randn(sum(n), 1, 64, generator=g)
    dev = c.cuda()
    bad_table = table.clone()
    bad_table[5, start[5] // PAGE] = total                    # a page outside the cache
    bad_table[6, start[6] // PAGE] = -1
    bad_start = list(start)
    bad_start[7] = -3                                         # outside the row
    bad_start[8] = 16 * table.shape[1]
    ws = put(v.cuda(), v.cuda(), bad_start, n, bad_table, dev, dict(base=1e4))
    assert pkg.read_status(ws) == 2
    good = [b for b in range(700) if b not in (5, 6, 7, 8)]
    cu = cu_of(n)
    keep = torch.cat([torch.arange(int(cu[b]), int(cu[b + 1])) for b in good])
    wv, wb = ref.append(v.double()[keep], [start[b] for b in good], cu_of([n[b] for b in good]), table[good], c.v, c.vs)
    for b in (5, 6):                                          # a second page of theirs that is fine is written
        if (start[b] % PAGE) + n[b] > PAGE:
            pytest.fail("choose sequences inside one page")
    got = [t.cpu() for t in dev]
    assert torch.equal(got[3], wb) and torch.equal(ref.e4m3_values(got[1]), wv)


@pytest.mark.parametrize("many", [0, 1200])
def test_append_reports_a_range_turned_round(many):
    """cu_n that falls: the sequence between is left out and reported, the others are written."""
    g = torch.Generator().manual_seed(8)
    n = [64, 0, 8] + [0] * many
    table, total = tables(g, [4, 1, 1] + [1] * many)
    c = Cache(g, total, 1, 64)
    v = torch.randn(72, 1, 64, generator=g)
    dev, good = c.cuda(), c.cuda()
    cu = torch.tensor([0, 64, 32, 40] + [40] * many, dtype=torch.int32, device="cuda")
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    args = (i32(table), ws, pkg.rope_spec(base=1e4))
    pkg.kvq_append(v.cuda(), v.cuda(), i32([0] * len(n)), cu, *dev, *args)
    assert pkg.read_status(ws) == 2
    order = torch.cat([v[:64], v[32:40]])
    assert pkg.read_status(put(order.cuda(), order.cuda(), [0] * len(n), n, table, good, dict(base=1e4))) == 0
    assert all(torch.equal(a, b) for a, b in zip(dev, good))


# ------------------------------------------------------------------- verify
def case(seed, lens, Bs, order, dtype, Hq, Hkv, hd, node=0, spec=None, sd=1.0, scale=None, lo=118, hi=122):
    g = torch.Generator().manual_seed(seed)
    per = 2 if order == "paired" else 1
    table, total = tables(g, [(L + PAGE - 1) // PAGE for L in lens])
    c = Cache(g, total, Hkv, hd, lo, hi)
    T = per * sum(Bs)
    q = (torch.randn(T, Hq, hd, generator=g) * sd).to(DT[dtype])
    kn, vn = (torch.randn(T, Hkv, hd, generator=g).to(DT[dtype]) for _ in range(2))
    tau = torch.cat([torch.randperm(b, generator=g) + 1 for b in Bs])
    return dict(q=q, c=c, table=table, kn=kn, vn=vn, tau=tau, lens=lens, Bs=Bs, cu=cu_of(Bs), order=order, node=node,
                spec=spec or dict(base=1e4), scale=scale or 1.0 / math.sqrt(hd), dtype=dtype)


ORDER = dict(paired=pkg.SIMSD_ORDER_PAIRED, nodes=pkg.SIMSD_ORDER_NODES, causal=pkg.SIMSD_ORDER_CAUSAL)


def launch(s, dev=None, out=None, ws=None, B_max=None, polls=0):
    if dev is None:
        dev = [t.cuda() for t in (s["q"], *s["c"].cuda(), s["kn"], s["vn"])]
    q, k, v, ks, vs, kn, vn = dev
    out = torch.empty(q.shape, dtype=q.dtype, device="cuda") if out is None else out
    args = (q, k, v, ks, vs, i32(s["table"]), kn, vn, i32(s["tau"]) if s["order"] == "paired" else None, i32(s["lens"]),
            i32(s["cu"]), out)
    total, top = int(s["cu"][-1]), B_max or max(s["Bs"])
    kw = dict(order=ORDER[s["order"]], node_size=s["node"])
    spec = pkg.rope_spec(**s["spec"])
    if ws is None:
        ws = torch.zeros(pkg.kvq_verify_workspace_size(*args, total, top, spec, s["scale"], **kw), dtype=torch.uint8, device="cuda")
    pkg.kvq_verify(*args, ws, total, top, spec, s["scale"], wait_polls=polls, **kw)
    return out, ws


def check(s, out):
    err = dict(f32=(0.0, 0.0), bf16=(2 * 2.0 ** -8, 2.0 ** -11))[s["dtype"]]
    want, off = ref.verify(s["q"], s["c"].k, s["c"].v, s["c"].ks, s["c"].vs, s["table"], s["kn"], s["vn"], s["tau"],
                           s["lens"], s["cu"], s["spec"], s["scale"], s["order"], s["node"], *err)
    off = off + want.abs() * torch.finfo(DT[s["dtype"]]).eps / 2 + 1e-30
    got = out.cpu().double()
    assert torch.equal(torch.isnan(got), torch.isnan(want))
    ok = ((got - want).abs() <= off) | torch.isnan(want)
    assert ok.all(), float(((got - want).abs() / off).nan_to_num().max())


LENS = [0, 1, 15, 16, 17, 127, 128, 129, 300, 513]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("order,Bs,node", [("paired", [1, 2, 3, 4, 5, 8, 4, 7, 1, 6], 0), ("nodes", [4, 8, 4, 16, 4, 4, 4, 12, 4, 8], 4),
                                           ("causal", [1, 3, 1, 7, 2, 1, 1, 5, 1, 9], 0)])
@pytest.mark.parametrize("Hq,Hkv,hd", [(8, 2, 128), (3, 3, 64), (7, 1, 128)])
def test_verify_matches_definition(dtype, order, Bs, node, Hq, Hkv, hd):
    s = case(Hq + hd, LENS, Bs, order, dtype, Hq, Hkv, hd, node)
    out, ws = launch(s)
    assert pkg.read_status(ws) == 0
    check(s, out)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("spec", [dict(base=1e4, interleaved=True), dict(base=1e6, rotary_dim=32),
                                  dict(base=1e6, rotary_dim=50, interleaved=True, scaling="ntk", factor=4.0),
                                  dict(base=1e6, rotary_dim=24), dict(base=1e6, scaling="yarn", factor=4.0, original_len=64),
                                  dict(base=1e6, scaling="banded", factor=8.0, original_len=256, fast=4.0, rotary_dim=64)])
def test_verify_rotary_forms(dtype, spec):
    for hd, order in ((128, "paired"), (64, "causal")):
        s = case(9, [40, 200, 3], [4, 2, 3], order, dtype, 4, 2, hd, 0, dict(spec))
        out, ws = launch(s)
        check(s, out)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("order,B,Hq,Hkv", [("paired", 32, 8, 2), ("causal", 64, 5, 1), ("nodes", 64, 2, 1), ("paired", 16, 4, 1),
                                            ("paired", 32, 7, 1)])
def test_verify_widest_sections(dtype, order, B, Hq, Hkv):
    """64 new tokens; one to four row tiles."""
    s = case(B + Hq, [70, 0, 260], [B, B, 8 if order == "nodes" else 3], order, dtype, Hq, Hkv, 128, 8 if order == "nodes" else 0)
    out, ws = launch(s)
    assert pkg.read_status(ws) == 0
    check(s, out)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("lens", [[5000], [4097, 100, 0, 2048], [3000] + [17] * 9])
def test_verify_key_splits(dtype, lens):
    """Few long sequences: the plan splits the keys, sequences shorter than a split among them."""
    s = case(len(lens), lens, [2] * len(lens), "paired", dtype, 4, 1, 64)
    out, ws = launch(s)
    assert ws.numel() > 256 and pkg.read_status(ws) == 0
    check(s, out)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("lens", [[300 - 7 * (i % 41) for i in range(60)], [200] * 60, [0] * 30 + [520] * 4 + [1] * 26,
                                  [5 * i % 97 for i in range(600)], [1025, 1100] * 4])
def test_verify_waves_and_cuts(dtype, lens):
    """More units than SMs: sequences in another order than the batch's, the last wave cut; a batch too large to be
    ordered; fewer units than SMs, cut in unequal pieces."""
    s = case(sum(lens), lens, [1] * len(lens), "causal", dtype, 8, 8, 64)
    out, ws = launch(s)
    assert pkg.read_status(ws) == 0
    check(s, out)


@pytest.mark.parametrize("B,Hq", [(16, 8), (8, 8), (4, 8), (12, 8)])
def test_verify_many_blocks(B, Hq):
    """Dozens of blocks a sequence, 128 to 32 rows: warps that drift apart, no wait that runs out, the same result twice."""
    s = case(B, [4000 - 300 * i for i in range(12)] * 4, [B] * 48, "paired", "bf16", Hq, 2, 128)
    dev = [t.cuda() for t in (s["q"], *s["c"].cuda(), s["kn"], s["vn"])]
    out, ws = launch(s, dev)
    for _ in range(20):
        assert torch.equal(launch(s, dev, ws=ws)[0], out)
    assert pkg.read_status(ws) == 0
    few = slice(0, 3)                                     # against 64 bits: the first sequences
    n = 2 * B * 3
    t = dict(s, lens=s["lens"][few], cu=s["cu"][:4], q=s["q"][:n], kn=s["kn"][:n], vn=s["vn"][:n], tau=s["tau"][:3 * B],
             table=s["table"][few])
    check(t, out[:n])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_verify_strided_rows(dtype):
    """q, k and v inside fused rows."""
    s = case(21, [33, 150], [4, 3], "causal", dtype, 4, 2, 128)
    T = 7
    rows = torch.cat([s["q"], s["kn"], s["vn"]], 1).cuda()
    q, kn, vn = rows[:, :4], rows[:, 4:6], rows[:, 6:]
    assert q.stride(0) == 8 * 128 and q.shape[0] == T
    c = s["c"].cuda()
    out, _ = launch(s, [q, *c, kn, vn], out=torch.empty(T, 4, 128, dtype=DT[dtype], device="cuda"))
    check(s, out)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_verify_ignores_what_lies_past_the_prompt(dtype):
    """NaN codes in the last page's unused slots and the pages after it, and NaN scales of pages not in the table."""
    s = case(22, [5, 130, 17], [2, 2, 2], "paired", dtype, 4, 2, 128)
    out, _ = launch(s)
    c = s["c"]
    used = torch.zeros(c.k.shape[0], dtype=torch.bool)
    for b, L in enumerate(s["lens"]):
        for j in range((L + PAGE - 1) // PAGE):
            used[s["table"][b, j]] = True
        if L % PAGE:
            c.k[s["table"][b, L // PAGE], :, L % PAGE:] = 0x7f
            c.v[s["table"][b, L // PAGE], :, L % PAGE:] = 0xff
    c.k[~used], c.v[~used], c.ks[~used], c.vs[~used] = 0x7f, 0x7f, 255, 255
    again, _ = launch(s)
    assert torch.equal(out, again)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_verify_marked_pages_read_as_nan(dtype):
    s = case(23, [40, 40], [1, 1], "paired", dtype, 2, 2, 64)
    s["c"].ks[s["table"][0, 1], 0] = 255
    s["c"].vs[s["table"][1, 2], 1] = 255
    out, _ = launch(s)
    bad = torch.isnan(out.float().cpu()).all(-1)
    # a section's rows of sequence 0 (head 0) and sequence 1 (head 1), nothing else
    assert torch.equal(bad, torch.tensor([[True, False], [True, False], [False, True], [False, True]]))
    assert torch.equal(torch.isnan(out.float().cpu()).any(-1), bad)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("order,B,Hq", [("paired", 4, 4), ("causal", 64, 2), ("nodes", 40, 6)])
def test_verify_odd_new_tokens_reach_the_rows_that_see_them(dtype, order, B, Hq):
    """NaN and infinite keys and values of a token: NaN in the rows that see it, no change in the others."""
    node = 8 if order == "nodes" else 0
    s = case(29, [50, 0], [B, B], order, dtype, Hq, 2, 128, node)
    clean, _ = launch(s)
    n = 2 * B if order == "paired" else B
    at = {0: 1, 1: n - 2}                                 # a token of each sequence, one head of it
    s["vn"][at[0], 0, 7], s["vn"][n + at[1], 1, 127] = math.nan, -math.inf
    s["kn"][at[1], 1, 5] = math.nan
    out, ws = launch(s)
    assert pkg.read_status(ws) == 0
    out, clean = out.cpu(), clean.cpu()
    for b, token, head in ((0, at[0], 0), (0, at[1], 1), (1, at[1], 1)):
        tau = s["tau"][b * B:(b + 1) * B] if order == "paired" else None
        sees = ref.visible(order, B, tau, node)[:, token]
        rows = out[b * n:(b + 1) * n, head * Hq // 2:(head + 1) * Hq // 2]
        same = clean[b * n:(b + 1) * n, head * Hq // 2:(head + 1) * Hq // 2]
        assert 0 < int(sees.sum()) < n
        assert torch.isnan(rows[sees]).all() and torch.equal(rows[~sees], same[~sees])
    assert torch.equal(out[n:, :Hq // 2], clean[n:, :Hq // 2])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("lo,hi,sd", [(63, 64, 1.0), (133, 135, 1e-4), (63, 135, 0.05), (118, 122, 60.0), (118, 122, 1e-6)])
def test_verify_scale_range_and_sharp_rows(dtype, lo, hi, sd):
    """Scales at both ends of their range and mixed, queries from tiny to ones whose softmax is one-hot."""
    s = case(24, [200, 31], [3, 2], "paired", dtype, 4, 2, 128, sd=sd, lo=lo, hi=hi)
    out, _ = launch(s)
    check(s, out)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_verify_one_large_score_and_many_small_ones(dtype):
    """A sink 12 above 4000 equal keys: their sum counts as much as the sink."""
    s = case(25, [4000], [1], "causal", dtype, 1, 1, 64)
    c, hd = s["c"], 64
    c.k[:], c.ks[:], c.vs[:] = 0, 127, 127
    q = torch.zeros(1, 1, hd)
    q[..., -1] = 8.0                                     # slowest pair: unrotated to 1e-3 at these positions
    s["q"] = q.to(DT[dtype])
    s["spec"] = dict(base=1e4, rotary_dim=2)
    c.k[s["table"][0, 0], 0, 3, -1] = 0x54               # 12 = 1.5 * 2^3
    s["scale"] = 0.125
    s["kn"] = torch.zeros_like(s["kn"])
    out, _ = launch(s)
    check(s, out)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_verify_bad_sequences_are_skipped(dtype):
    s = case(26, [20, 33, 48, 16], [2, 2, 2, 2], "nodes", dtype, 4, 2, 64, node=2)
    good, _ = launch(s)
    s["lens"] = [20, -1, 16 * s["table"].shape[1] + 1, 16]
    out = torch.full(s["q"].shape, 7.0, dtype=DT[dtype], device="cuda")
    out, ws = launch(s, out=out)
    assert pkg.read_status(ws) == 2
    assert torch.equal(out[:2], good[:2]) and torch.equal(out[6:], good[6:]) and (out[2:6] == 7).all()
    s["lens"] = [20, 33, 48, 16]
    s["table"][1, 1] = s["c"].k.shape[0]                  # a page outside the cache counts as absent
    s["table"][2, 0] = -1
    out, ws = launch(s)
    assert pkg.read_status(ws) == 2
    assert torch.isfinite(out.float()).all() and torch.equal(out[:2], good[:2]) and torch.equal(out[6:], good[6:])


def test_verify_two_graphs_and_streams():
    """Two captured calls with a workspace each, replayed at once on two streams, give what eager calls give."""
    runs = []
    for i in range(2):
        s = case(30 + i, [700 + 5000 * i, 20], [4, 4], "paired", "bf16", 8, 2, 128)
        dev = [t.cuda() for t in (s["q"], *s["c"].cuda(), s["kn"], s["vn"])]
        want, ws = launch(s, dev)
        args = (*dev[:5], i32(s["table"]), dev[5], dev[6], i32(s["tau"]), i32(s["lens"]), i32(s["cu"]), torch.zeros_like(want))
        spec = pkg.rope_spec(**s["spec"])
        graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
        with torch.cuda.graph(graph, stream=side):
            pkg.kvq_verify(*args, ws, 8, 4, spec, s["scale"])
        runs.append((graph, side, args[-1], want, (args, ws)))     # the graph's memory stays alive
    torch.cuda.synchronize()
    for _ in range(3):
        for graph, side, _, _, _ in runs:
            with torch.cuda.stream(side):
                graph.replay()
    torch.cuda.synchronize()
    for _, _, out, want, _ in runs:
        assert torch.equal(out, want)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("seqs", [2, 50])
def test_verify_captured_behind_copies_and_joins(dtype, seqs):
    """In a graph right behind a copy, behind a join of two streams, and twice in a row: what an eager call gives."""
    s = case(36, [100 - i for i in range(seqs)], [2] * seqs, "causal", dtype, 8, 8, 64)
    q, *rest = [t.cuda() for t in (s["q"], *s["c"].cuda(), s["kn"], s["vn"])]
    want, ws = launch(s, [q, *rest])
    qs, outs = torch.zeros_like(q), [torch.zeros_like(want) for _ in range(3)]
    table, lens, cu, spec = i32(s["table"]), i32(s["lens"]), i32(s["cu"]), pkg.rope_spec(**s["spec"])
    wss = [torch.zeros_like(ws) for _ in range(2)]

    def call(out, w):
        pkg.kvq_verify(qs, *rest[:4], table, *rest[4:], None, lens, cu, out, w, 2 * seqs, 2, spec, s["scale"], order=ORDER["causal"])

    graph, side, other = torch.cuda.CUDAGraph(), torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=side):
        qs.copy_(q)
        call(outs[0], wss[0])
        other.wait_stream(side)
        with torch.cuda.stream(other):
            call(outs[1], wss[1])
        call(outs[0], wss[0])
        side.wait_stream(other)
        call(outs[2], wss[0])
        qs.zero_()
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for o in outs)
    assert all(pkg.read_status(w) == 0 for w in wss)


def test_append_and_verify_captured_in_several_waves():
    """Sequences taken by length, the last wave cut, in a graph behind the append that their last pages come from."""
    s = case(33, [397 - 8 * i for i in range(40)], [1] * 40, "causal", "bf16", 8, 8, 64)
    q, *cache, kn, vn = (t.cuda() for t in (s["q"], *s["c"].cuda(), s["kn"], s["vn"]))
    before = [t.clone() for t in cache]
    table, lens, cu, start = i32(s["table"]), i32(s["lens"]), i32(s["cu"]), i32([16 * (L // 16) for L in s["lens"]])
    spec, out = pkg.rope_spec(**s["spec"]), torch.empty_like(q)
    args = (q, *cache, table, kn, vn, None, lens, cu, out)
    n = pkg.kvq_verify_workspace_size(*args, 40, 1, spec, s["scale"], order=ORDER["causal"])
    ws, wsv = (torch.zeros(m, dtype=torch.uint8, device="cuda") for m in (256, n))

    def step():
        pkg.kvq_append(kn, vn, start, cu, *cache, table, ws, spec)
        pkg.kvq_verify(*args, wsv, 40, 1, spec, s["scale"], order=ORDER["causal"])

    step()
    want, after = out.clone(), [t.clone() for t in cache]
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=side):
        step()
    for _ in range(2):
        out.fill_(7)
        for t, old in zip(cache, before):
            t.copy_(old)
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want) and all(torch.equal(t, a) for t, a in zip(cache, after))
    assert pkg.read_status(ws) == 0 and pkg.read_status(wsv) == 0


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_cache_of_more_than_32_bits(dtype):
    """Pages and rows whose offsets pass 2^32 elements: the same codes and results as at the front."""
    Hkv, hd, far = 8, 128, 2 ** 32 // (8 * 16 * 128) + 3
    s = case(34, [70], [4], "paired", dtype, 8, Hkv, hd)
    spec, n = pkg.rope_spec(**s["spec"]), 70
    g = torch.Generator().manual_seed(35)
    k, v = (torch.randn(n, Hkv, hd, generator=g).to(DT[dtype]).cuda() for _ in range(2))
    shape = (far + 5, Hkv, PAGE, hd)
    kc, vc = (torch.zeros(shape, dtype=torch.uint8, device="cuda") for _ in range(2))
    ks, vs = (torch.zeros(shape[:2], dtype=torch.uint8, device="cuda") for _ in range(2))
    q, kn, vn = s["q"].cuda(), s["kn"].cuda(), s["vn"].cuda()
    outs, stride = [], 2 ** 25 + 8 * hd                   # 70 rows of it pass 2^31 elements
    wide = torch.zeros(n, stride, dtype=DT[dtype], device="cuda")
    wide[:, :Hkv * hd] = k.flatten(1)
    for at, rows in ((0, k), (far, wide[:, :Hkv * hd].unflatten(1, (Hkv, hd)))):
        table = torch.arange(at, at + 5)[None]
        ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
        pkg.kvq_append(rows, v, i32([0]), i32([0, n]), kc, vc, ks, vs, i32(table), ws, spec)
        s["table"] = table
        outs.append(launch(s, [q, kc, vc, ks, vs, kn, vn]))
        assert pkg.read_status(ws) == 0 and pkg.read_status(outs[-1][1]) == 0
    assert torch.equal(outs[0][0], outs[1][0]) and int(ks[far].max()) > 0
    for t in (kc, vc, ks, vs):
        assert torch.equal(t[:5], t[far:])


def test_step_of_the_loop():
    """Requests admitted, their prompts appended, a verification pass, the kept tokens appended behind it, and the next
    pass: every stage fed by the one before, against the same chain in 64 bits on the cache's own values."""
    g = torch.Generator().manual_seed(40)
    Hq, Hkv, hd, B, batch, width, cap = 4, 2, 128, 4, 3, 8, 30
    spec = dict(base=1e4, rotary_dim=64)
    lens0 = [37, 5, 64]
    free, queue = i32(torch.randperm(cap, generator=g)), i32([0, cap])
    table, held = i32(torch.zeros(batch, width)), i32([0] * batch)
    served, ws_map = i32([0] * batch), torch.zeros(256, dtype=torch.uint8, device="cuda")
    c = Cache(g, cap, Hkv, hd)
    dev = c.cuda()
    state = [c.k, c.v, c.ks, c.vs]

    def both(k, v, start, n, take=None):
        put(k.cuda(), v.cuda(), start, n, table.cpu(), dev, spec, take)
        pos = torch.cat([torch.arange(s, s + m) for s, m in zip(start, n)])
        cu = cu_of(n)
        wv, wvb = ref.append(v.double(), start, cu, table.cpu(), state[1], state[3], take)
        wk, wkb = ref.append(ref.rope(k, pos, spec), start, cu, table.cpu(), state[0], state[2], take)
        got = [t.cpu() for t in dev]
        assert torch.equal(got[3], wvb) and torch.equal(ref.e4m3_values(got[1]), wv)
        check_keys(got[0], got[2], None, None, wk, wkb)
        state[:] = got

    pkg.page_map(i32(lens0), None, held, queue, free, table, held, queue, served, None, ws_map, 0)
    assert served.tolist() == [1, 1, 1] and held.tolist() == [3, 1, 4]
    N = sum(lens0)
    both(torch.randn(N, Hkv, hd, generator=g).bfloat16(), torch.randn(N, Hkv, hd, generator=g).bfloat16(), [0] * batch, lens0)
    lens = list(lens0)
    for step in range(2):
        s = case(50 + step, lens, [B] * batch, "paired", "bf16", Hq, Hkv, hd, spec=spec)
        s["c"].k, s["c"].v, s["c"].ks, s["c"].vs = state
        s["table"] = table.cpu().long()
        out, ws = launch(s, [s["q"].cuda(), *dev, s["kn"].cuda(), s["vn"].cuda()])
        assert pkg.read_status(ws) == 0
        check(s, out)
        # sequences 0 and 2 close their block: B tokens of the data section stay
        keep = [B, 0, B]
        slots = torch.empty(2 * B * batch, dtype=torch.int64, device="cuda")
        pkg.page_map(i32(lens), i32(cu_of(keep)), held, queue, free, table, held, queue, served, slots, ws_map, 2 * B * batch)
        for i, (b, p) in enumerate([(b, lens[b] + j) for b in range(batch) for j in range(keep[b])]):
            assert int(slots[i]) == int(table[b, p // PAGE]) * PAGE + p % PAGE
        both(s["kn"], s["vn"], lens, [2 * B] * batch, keep)
        lens = [L + m for L, m in zip(lens, keep)]
    assert pkg.read_status(ws_map) == 0


def test_verify_timeout_writes_nothing():
    """wait_polls < 0 gives up at once: the timeout bit, out untouched, and the workspace good for the next call."""
    s = case(60, [300, 40], [4, 4], "paired", "bf16", 8, 2, 128)
    want, ws = launch(s)
    out = torch.full_like(want, 7.0)
    launch(s, out=out, ws=ws, polls=-1)
    assert pkg.read_status(ws) & 1
    assert (out == 7).all()
    again, _ = launch(s, ws=ws)
    assert pkg.read_status(ws) == 0 and torch.equal(again, want)
