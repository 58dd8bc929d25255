"""simsd_kv4_append, _read and _verify against their 64-bit forms (kv4_ref).

Append.  A scale is the one nearest to amax / 6, a code the one nearest to x /
scale.  Values are quantised as they come, so their bytes must be equal.  A
rotated key is fp32 in the kernel, off by at most 2e-6 of its row's largest
element (angles of 3e-7 rad, three roundings of 2^-24 for each of two
products), so its code or scale may be the neighbour where the exact value lies
that close to the middle.

Read.  Exact (e4m3: rounded once).

Verify.  kv4_ref.verify gives each element's bound: query elements, new keys,
new values and weights off by 2^-11 of themselves (f16; fp32 data: none), then
the output's own rounding, half a step."""
import math

import pytest
import torch

import kv4_ref as ref
import kvq_ref
import speculative_decoding_diffusion_gb300 as pkg

pytestmark = pytest.mark.gpu
PAGE = 16
DT = {"f32": torch.float32, "bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn}
ORDER = {"paired": pkg.SIMSD_ORDER_PAIRED, "nodes": pkg.SIMSD_ORDER_NODES, "causal": pkg.SIMSD_ORDER_CAUSAL}
ROPES = [dict(base=1e4), dict(base=1e4, interleaved=True, rotary_dim=32), dict(base=1e6, rotary_dim=48, scaling="linear", factor=2.0),
         dict(base=1e6, rotary_dim=50), dict(base=1e6, rotary_dim=32), dict(base=1e5, scaling="yarn", factor=4.0, original_len=64)]


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


def make_cache(gen, pages, heads, hd, lo=0x68, hi=0x80):
    """Random records: any codes, scales of 2^-2 to 2 or so."""
    rec = torch.randint(0, 256, (pages, heads, 18 * hd), generator=gen).to(torch.uint8)
    rec[..., 16 * hd:] = torch.randint(lo, hi, (pages, heads, 2 * hd), generator=gen).to(torch.uint8)
    return rec


def workspace(n=256):
    return torch.zeros(n, dtype=torch.uint8, device="cuda")


def put(k, v, start, n, table, cache, spec, take=None):
    ws = workspace()
    pkg.kv4_append(k, v, i32(start), i32(cu_of(n)), cache, i32(table), ws, pkg.rope_spec(**spec),
                   take=None if take is None else i32(take))
    return ws


def check_keys(got, want, x, slots):
    """Codes and scales of rotated keys x [N, H, hd]: nearest up to the rotation's error; slots: where each row lies."""
    gk, gb, _, _ = ref.unpack(got)
    wk, wb, _, _ = ref.unpack(want)
    flips = 0
    for r, (page, i) in enumerate(slots):
        tol = 2e-6 * x[r].abs().amax(-1, keepdim=True)                        # [H, 1]
        top = x[r].unflatten(-1, (-1, 16)).abs().amax(-1)
        s, best = ref.scale_values(gb[page, :, i]), ref.scale_values(wb[page, :, i])
        assert ((s - top / 6).abs() <= (best - top / 6).abs() + 2 * tol / 6).all()
        every = torch.cat([ref.CODES, -ref.CODES]) * s[..., None, None]       # [H, groups, 1, 16]
        g = x[r].unflatten(-1, (-1, 16))
        near = (every - g[..., None]).abs().amin(-1).flatten(-2)
        off = (ref.values(gk[page, :, i], gb[page, :, i]) - x[r]).abs()
        assert (off <= near + 2 * tol).all()
        flips += int((gk[page, :, i] != wk[page, :, i]).sum())
    assert flips <= 1e-3 * x.numel()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("hd,H", [(128, 2), (64, 9)])
@pytest.mark.parametrize("spec", ROPES)
def test_append_matches_definition(dtype, hd, H, spec):
    g = torch.Generator().manual_seed(hd + H)
    start = [0, 5, 16, 31, 100, 7, 0, 15, 14]
    n = [33, 1, 16, 2, 47, 0, 1, 17, 1]
    table, total = tables(g, [(s + m + PAGE - 1) // PAGE for s, m in zip(start, n)])
    cache = make_cache(g, total, H, hd)
    N = sum(n)
    k = (torch.randn(N, H, hd, generator=g) * torch.exp2(torch.randint(-3, 4, (N, H, 1), generator=g).float())).to(DT[dtype])
    v = (torch.randn(N, H, hd, generator=g) * 3).to(DT[dtype])
    dev = cache.cuda()
    ws = put(k.cuda(), v.cuda(), start, n, table, dev, spec)
    assert pkg.read_status(ws) == 0
    cu = cu_of(n)
    pos = torch.cat([torch.arange(s, s + m) for s, m in zip(start, n)])
    seq = torch.repeat_interleave(torch.arange(len(n)), torch.tensor(n))
    x = kvq_ref.rope(k, pos, spec)
    want = ref.append(ref.append(cache, 1, v.double(), start, cu, table), 0, x, start, cu, table)
    got = dev.cpu()
    assert torch.equal(got[..., 8 * hd:16 * hd], want[..., 8 * hd:16 * hd])   # value codes
    assert torch.equal(got[..., 17 * hd:], want[..., 17 * hd:])               # and scales
    slots = [(int(table[b, p // PAGE]), int(p % PAGE)) for b, p in zip(seq.tolist(), pos.tolist())]
    check_keys(got, want, x, slots)
    # what no token of the call owns is as it was: with the keys of the call put back, all bytes are equal
    gk, gb, _, _ = ref.unpack(got)
    wk, wb, _, _ = ref.unpack(want)
    mine = torch.zeros(total, PAGE, dtype=torch.bool)
    for p, i in slots:
        mine[p, i] = True
    m = mine[:, None, :, None]
    assert torch.equal(gk.masked_fill(m, 0), wk.masked_fill(m, 0)) and torch.equal(gb.masked_fill(m, 0), wb.masked_fill(m, 0))
    # the same call again finds the same state
    dev2 = dev.clone()
    put(k.cuda(), v.cuda(), start, n, table, dev2, spec)
    assert torch.equal(dev, dev2)


def test_append_borders_zeros_and_the_unfinite():
    """Middles between scales and between codes, zeros, the range's ends; a NaN or an infinity marks its group alone."""
    hd, spec = 64, dict(base=1e4, rotary_dim=2)                               # elements 2.. pass unrotated
    mids = ((ref.SCALES[1:] + ref.SCALES[:-1]) / 2 * 6)[::7].tolist()
    tops = mids + [0.0, -0.0, 6.0, 2.0 ** -20, 6 * 2.0 ** -18, 1e-38, 61440.0, 65000.0, 3e38]
    rows = torch.zeros(len(tops), 1, hd)
    ties = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, -0.25, -5.0, 0.2500001, 4.9999995])
    for i, t in enumerate(tops):
        rows[i, 0, 16] = t                                                    # group 1: its largest magnitude
        s = float(ref.scale_values(ref.scale_bytes(rows[i].double()))[0, 1])
        rows[i, 0, 17:17 + len(ties)] = ties * s
        rows[i, 0, 40] = 1.0                                                  # group 2: of its own
    odd = torch.zeros(4, 1, hd)
    odd[:, 0, 16:48] = torch.randn(32, generator=torch.Generator().manual_seed(4))
    odd[0, 0, 20], odd[1, 0, 31], odd[2, 0, 47], odd[3, 0, 16] = math.nan, math.inf, -math.inf, math.nan
    x = torch.cat([rows, odd])
    N = len(x)
    table, total = tables(torch.Generator().manual_seed(1), [(N + 15) // 16 + 1])
    cache = make_cache(torch.Generator().manual_seed(2), total, 1, hd)
    dev = cache.cuda()
    ws = put(x.cuda(), x.cuda(), [3], [N], table, dev, spec)
    assert pkg.read_status(ws) == 0
    want = ref.append(ref.append(cache, 1, x.double(), [3], cu_of([N]), table), 0, x.double(), [3], cu_of([N]), table)
    for a, b, name in zip(ref.unpack(dev.cpu()), ref.unpack(want), ("kc", "kb", "vc", "vb")):
        if name[1] == "b":
            assert torch.equal(a, b), name
        else:                                                                 # (the codes of a marked group say nothing)
            nan = (ref.unpack(want)[1 if name[0] == "k" else 3] == ref.NAN_BYTE).repeat_interleave(16, -1)
            assert torch.equal(ref.values(a, torch.full_like(a[..., ::16], 0x78)).masked_fill(nan, 0),
                               ref.values(b, torch.full_like(b[..., ::16], 0x78)).masked_fill(nan, 0)), name


def test_append_takes_the_first_rows_and_strides():
    g = torch.Generator().manual_seed(9)
    hd, H, start, n, take = 128, 3, [4, 0, 33], [5, 7, 20], [5, 0, 11]
    table, total = tables(g, [3, 3, 4])
    cache = make_cache(g, total, H, hd)
    N = sum(n)
    qkv = torch.randn(N, 2 * H + 4, hd, generator=g).bfloat16()
    k, v = qkv[:, 4:4 + H], qkv[:, 4 + H:]
    dev, dev2 = cache.cuda(), cache.cuda()
    qd = qkv.cuda()
    spec = dict(base=1e4)
    assert pkg.read_status(put(qd[:, 4:4 + H], qd[:, 4 + H:], start, n, table, dev, spec, take)) == 0
    put(k.contiguous().cuda(), v.contiguous().cuda(), start, n, table, dev2, spec, take)
    assert torch.equal(dev, dev2)
    want = ref.append(cache, 1, v.double(), start, cu_of(n), table, take)
    assert torch.equal(dev.cpu()[..., 8 * hd:16 * hd], want[..., 8 * hd:16 * hd])


def test_append_and_read_bad_inputs():
    """Sequences whose numbers are out of range leave the others alone and set the bit."""
    g = torch.Generator().manual_seed(3)
    hd, H = 64, 2
    start, n = [0, 5, -1, 60, 3], [4, 3, 2, 9, 6]                             # sequence 2: start < 0; 3: past its row
    table, total = tables(g, [4] * 5)
    table[4, 0] = total + 7                                                   # no such page
    cache = make_cache(g, total, H, hd)
    x = torch.randn(sum(n), H, hd, generator=g)
    dev = cache.cuda()
    ws = put(x.cuda(), x.cuda(), start, n, table, dev, dict(base=1e4, rotary_dim=2))
    assert pkg.read_status(ws) == 2
    good = [4, 3, 0, 0, 0]
    want = ref.append(cache, 1, x.double(), [0, 5, 0, 0, 0], cu_of(n), table, good)
    assert torch.equal(dev.cpu()[..., 8 * hd:16 * hd], want[..., 8 * hd:16 * hd])
    out = torch.full((sum(n), H, hd), 7.0, device="cuda")
    k, v = out.clone(), out.clone()
    ws = workspace()
    pkg.kv4_read(dev, i32(table), i32(start), i32(cu_of(n)), k, v, ws)
    assert pkg.read_status(ws) == 2
    assert (k[7:] == 7).all() and (v[7:] == 7).all() and not (v[:7] == 7).all()
    for cu in ([0, 4, 3, 9, 18, 24], [0, 4, 7, 9, 18, 25], [-1, 4, 7, 9, 18, 24]):
        ws = workspace()
        pkg.kv4_append(x.cuda(), x.cuda(), i32([0] * 5), i32(cu), dev, i32(table), ws, pkg.rope_spec())
        assert pkg.read_status(ws) == 2
    # rows before the first sequence's and behind the last one's are no bad input
    ws = workspace()
    before = dev.clone()
    pkg.kv4_append(x.cuda(), x.cuda(), i32([0]), i32([3, 3]), dev, i32(table[:1]), ws, pkg.rope_spec())
    assert pkg.read_status(ws) == 0 and torch.equal(before, dev)


@pytest.mark.parametrize("batch", [1, 31, 33, 700])
def test_rows_find_their_sequences(batch):
    """Empty sequences among others, batches of one, two and three steps of the search."""
    g = torch.Generator().manual_seed(batch)
    n = torch.randint(0, 4, (batch,), generator=g)
    n[torch.rand(batch, generator=g) < 0.3] = 0
    n[-1] = 2
    start = torch.randint(0, 20, (batch,), generator=g)
    table, total = tables(g, [2] * batch)
    cache = make_cache(g, total, 1, 64)
    v = torch.empty(int(n.sum()), 1, 64, device="cuda")
    ws = workspace()
    pkg.kv4_read(cache.cuda(), i32(table), i32(start), i32(cu_of(n)), None, v, ws)
    assert pkg.read_status(ws) == 0
    want = torch.cat([ref.rows(cache, table, b, int(start[b]), int(n[b]))[1] for b in range(batch)])
    assert torch.equal(v.double().cpu(), want)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "e4m3"])
@pytest.mark.parametrize("hd,H", [(128, 3), (64, 1)])
def test_read_is_exact(dtype, hd, H):
    g = torch.Generator().manual_seed(hd)
    start, n = [0, 5, 16, 31, 100, 7, 15], [33, 1, 16, 2, 47, 0, 18]
    table, total = tables(g, [(s + m + PAGE - 1) // PAGE for s, m in zip(start, n)])
    cache = make_cache(g, total, H, hd, 0, 0xe3)                              # every scale of the range
    cache[::2, :, 16 * hd:][..., ::5] = ref.NAN_BYTE
    cu, N = cu_of(n), sum(n)
    want = [torch.cat([ref.rows(cache, table, b, start[b], n[b])[i] for b in range(len(n))]) for i in (0, 1)]
    fused = torch.zeros(N + 2, 2 * H + 1, hd, device="cuda").to(DT[dtype])    # rows of a wider tensor, two behind the last
    for kv in ((True, True), (True, False), (False, True)):
        fused.view(torch.uint8).fill_(0x11)
        k, v = fused[:, :H], fused[:, H:2 * H]
        ws = workspace()
        pkg.kv4_read(cache.cuda(), i32(table), i32(start), i32(cu), k if kv[0] else None, v if kv[1] else None, ws)
        assert pkg.read_status(ws) == 0
        raw = fused.view(torch.uint8).view(N + 2, 2 * H + 1, -1)
        assert (raw[:, 2 * H:] == 0x11).all() and (raw[N:] == 0x11).all()
        for i, t in enumerate((k, v)):
            if not kv[i]:
                assert (t.view(torch.uint8) == 0x11).all()
                continue
            got = t[:N].float().double().cpu()
            w = kvq_ref.code(want[i]) if dtype == "e4m3" else want[i]
            w = torch.where(torch.isfinite(want[i]), w, math.nan)
            assert torch.equal(got.isnan(), w.isnan()) and torch.equal(got.nan_to_num(0), w.nan_to_num(0))


def verify(q, cache, table, kn, vn, tau, lens, cu, B_max, spec, scale, order, node=0, wait_polls=0, ws=None, out=None):
    out = torch.full(q.shape, 7.0, dtype=q.dtype, device="cuda") if out is None else out
    args = (q, cache, i32(table), kn, vn, tau, i32(lens), i32(cu), out)
    rope = pkg.rope_spec(**spec)
    size = pkg.kv4_verify_workspace_size(*args, int(cu[-1]), B_max, rope, scale, order=ORDER[order], node_size=node)
    ws = workspace(size) if ws is None else ws
    pkg.kv4_verify(*args, ws, int(cu[-1]), B_max, rope, scale, order=ORDER[order], node_size=node, wait_polls=wait_polls)
    return out, ws


def close(got, want, off, dtype):
    half = 2.0 ** -8 if dtype == "bf16" else 2.0 ** -24
    got = got.double().cpu()
    assert torch.equal(got.isnan(), want.isnan())
    bad = ~((got - want).abs() <= off + half * want.abs() + 1e-30) & ~want.isnan()
    assert not bad.any(), ((got - want).abs() / (off + half * want.abs() + 1e-30)).nan_to_num(0).max()


def case(seed, lens, Bs, order, dtype, G, Hkv, hd, spare_nan=True):
    g = torch.Generator().manual_seed(seed)
    per = 2 if order == "paired" else 1
    table, total = tables(g, [(P + PAGE - 1) // PAGE for P in lens])
    cache = make_cache(g, total, Hkv, hd)
    if spare_nan:                                                             # slots past a prompt's end hold anything
        for b, P in enumerate(lens):
            if P % PAGE:
                _, _, s = ref.places(hd)[0]
                _, _, sv = ref.places(hd)[1]
                rec = cache[int(table[b, P // PAGE])]
                rec[:, s[P % PAGE:].flatten()] = 0xff
                rec[:, sv[P % PAGE:].flatten()] = 0xff
    cu = cu_of(Bs)
    T = per * int(cu[-1])
    q = torch.randn(T, G * Hkv, hd, generator=g).to(DT[dtype])
    kn, vn = (torch.randn(T, Hkv, hd, generator=g).to(DT[dtype]) for _ in range(2))
    tau = torch.cat([torch.randperm(B, generator=g) + 1 for B in Bs])
    return cache, table, cu, q, kn, vn, tau


LENS = [(0, 1, 15, 16, 17), (33, 129, 0, 511), (1000,), (300, 64)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("order,Bs,node", [("causal", (1,), 0), ("causal", (3, 1, 5), 0), ("causal", (64, 17), 0),
                                           ("paired", (4, 4), 0), ("paired", (1, 8, 3), 0), ("paired", (32, 5), 0),
                                           ("nodes", (4, 8), 4), ("nodes", (64, 32), 32), ("nodes", (5, 10), 5)])
@pytest.mark.parametrize("G,Hkv,hd", [(4, 2, 128), (1, 3, 64), (7, 1, 128), (8, 2, 64)])
def test_verify_matches_definition(dtype, order, Bs, node, G, Hkv, hd):
    i = (len(order) + len(Bs) + G) % len(LENS)
    lens = LENS[i]
    Bs = [Bs[j % len(Bs)] for j in range(len(lens))]
    spec = ROPES[(G + hd + len(Bs)) % len(ROPES)]
    cache, table, cu, q, kn, vn, tau = case(i, lens, Bs, order, dtype, G, Hkv, hd)
    scale = 1 / math.sqrt(hd)
    out, ws = verify(q.cuda(), cache.cuda(), table, kn.cuda(), vn.cuda(), i32(tau), lens, cu, max(Bs), spec, scale, order, node)
    assert pkg.read_status(ws) == 0
    want, off = ref.verify(q, cache, table, kn, vn, tau, lens, cu, spec, scale, order, node, 2.0 ** -11 if dtype == "bf16" else 0.0)
    close(out, want, off, dtype)


@pytest.mark.parametrize("B", [1, 2, 4, 8, 16])
def test_verify_split_keys(B):
    """Few long prompts: the keys of a unit go to several SMs and are merged; a short one beside a long one."""
    lens = (6000, 37, 2500)
    spec = dict(base=1e6)
    cache, table, cu, q, kn, vn, tau = case(B, lens, [B] * 3, "paired", "bf16", 4, 1, 128)
    out, ws = verify(q.cuda(), cache.cuda(), table, kn.cuda(), vn.cuda(), i32(tau), lens, cu, B, spec, 0.1, "paired")
    assert pkg.read_status(ws) == 0 and ws.numel() > 3 * 2 * B * 4 * 128 * 4
    want, off = ref.verify(q, cache, table, kn, vn, tau, lens, cu, spec, 0.1, "paired", 0, 2.0 ** -11)
    close(out, want, off, "bf16")


@pytest.mark.parametrize("B", [1, 4, 16])
def test_verify_sizes_of_rows_and_values(B):
    """Peaked scores that grow along the keys (references move), tiny and huge queries, values and new tokens."""
    lens = (700, 90)
    cache, table, cu, q, kn, vn, tau = case(50 + B, lens, [B] * 2, "causal", "bf16", 4, 2, 128)
    hd = 128
    for j in range(int((lens[0] + 15) // 16)):                                # scales of keys rise with the position
        cache[int(table[0, j]), :, 16 * hd:17 * hd] = min(0x58 + j, 0x88)
    q = (q.float() * torch.exp2(torch.arange(q.shape[1]).float() * 3 - 12)[None, :, None]).bfloat16()
    vn = (vn.float() * torch.exp2(torch.arange(vn.shape[0]).float() * 5 - 30)[:, None, None]).bfloat16()
    kn = (kn.float() * torch.exp2(-torch.arange(kn.shape[0]).float())[:, None, None]).bfloat16()
    spec = dict(base=1e4)
    out, ws = verify(q.cuda(), cache.cuda(), table, kn.cuda(), vn.cuda(), None, lens, cu, B, spec, 0.05, "causal")
    assert pkg.read_status(ws) == 0
    want, off = ref.verify(q, cache, table, kn, vn, tau, lens, cu, spec, 0.05, "causal", 0, 2.0 ** -11)
    # each of the up to 716 products may be off by 2^-32 of the row's largest, which is at most the result's largest
    # element times the sum of weights
    off = off + 716 * 2.0 ** -32 * want.abs().amax(-1, keepdim=True) * 2
    close(out, want, off, "bf16")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("B", [2, 6, 16])
def test_verify_unfinite_values_reach_who_sees_them(dtype, B):
    """A new token's NaN or infinity, a marked group: NaN for the rows that see it, nothing for the others."""
    lens = (40, 70)
    cache, table, cu, q, kn, vn, tau = case(B, lens, [B] * 2, "paired", dtype, 4, 1, 128)
    hd = 128
    vn[B - 1, 0, 3], kn[2 * B - 1, 0, 5] = math.inf, math.nan                 # D_B's value, D~_B's key, of sequence 0
    cache[int(table[1, 1]), 0, 17 * hd + 2 * 3 + 1] = ref.NAN_BYTE            # sequence 1, position 17, value group 3
    spec = dict(base=1e4)
    args = (table, kn.cuda(), vn.cuda(), i32(tau), lens, cu, B, spec, 0.1, "paired")
    out, ws = verify(q.cuda(), cache.cuda(), *args)
    assert pkg.read_status(ws) == 0
    see = kvq_ref.visible("paired", B, tau[:B], 0)
    hit = (see[:, B - 1] | see[:, 2 * B - 1])
    got = out.float().cpu()
    assert got[:2 * B][hit].isnan().all() and not got[:2 * B][~hit].isnan().any()
    assert got[2 * B:, :, 48:64].isnan().all() and not got[2 * B:, :, :48].isnan().any() and not got[2 * B:, :, 64:].isnan().any()
    vn[B - 1, 0, 3], kn[2 * B - 1, 0, 5] = 0.5, 0.5                           # the others: the same without it
    out2, _ = verify(q.cuda(), cache.cuda(), table, kn.cuda(), vn.cuda(), *args[3:])
    assert torch.equal(out[:2 * B][~hit.cuda()], out2[:2 * B][~hit.cuda()])
    # a marked key group: the row is NaN
    cache[int(table[1, 0]), 0, 16 * hd + 8 * 4 + 1] = ref.NAN_BYTE
    out, _ = verify(q.cuda(), cache.cuda(), table, kn.cuda(), vn.cuda(), *args[3:])
    assert out[2 * B:].isnan().all() and not out[:2 * B].isnan().any()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("B", [1, 16])
def test_verify_bad_inputs(dtype, B):
    """Each bad sequence sets the bit and is left out; the others' rows are right."""
    lens = [40, 70, 33, 1000, 50]
    cache, table, cu, q, kn, vn, tau = case(7, [40, 70, 33, 16, 50], [B] * 5, "causal", dtype, 4, 1, 64)
    spec = dict(base=1e4)
    want, off = ref.verify(q, cache, table, kn, vn, tau, [40, 70, 33, 16, 50], cu, spec, 0.1, "causal", 0,
                           2.0 ** -11 if dtype == "bf16" else 0.0)
    bad = table.clone()
    bad[2, 1] = -3                                                            # a page that does not exist counts as absent
    out, ws = verify(q.cuda(), cache.cuda(), bad, kn.cuda(), vn.cuda(), None, lens, cu, B, spec, 0.1, "causal")
    assert pkg.read_status(ws) == 2
    ok = [0, 1, 4]
    rows = torch.cat([torch.arange(b * B, (b + 1) * B) for b in ok])
    close(out[rows.cuda()], want[rows], off[rows], dtype)
    assert (out[3 * B:4 * B] == 7).all()
    # sequence 2: the same as with keys 16.. masked, i.e. a causal row over the other keys; compare with 64 bits
    s = slice(2 * B, 3 * B)
    assert torch.isfinite(out[s].float()).all() and not (out[s] == 7).any()
    cu2 = cu.clone()
    cu2[2] = cu2[1]                                                           # B = 0, and one of 2 B
    out, ws = verify(q.cuda(), cache.cuda(), table, kn.cuda(), vn.cuda(), None, [40, 70, 33, 16, 50], cu2, B, spec, 0.1, "causal")
    assert pkg.read_status(ws) == 2
    close(out[:B], want[:B], off[:B], dtype)


@pytest.mark.parametrize("B,lens", [(1, (900, 20)), (16, (900, 20)), (4, (0, 5))])
def test_verify_waits_that_give_up(B, lens):
    """wait_polls < 0: every wait gives up at once; the bit is set and the next call is right."""
    cache, table, cu, q, kn, vn, tau = case(B, lens, [B] * 2, "paired", "bf16", 4, 2, 128)
    spec = dict(base=1e4)
    args = (q.cuda(), cache.cuda(), table, kn.cuda(), vn.cuda(), i32(tau), lens, cu, B, spec, 0.1, "paired")
    _, ws = verify(*args, wait_polls=-1)
    assert pkg.read_status(ws) == 1                                           # (there are keys to wait for)
    out, ws = verify(*args, ws=ws)
    assert pkg.read_status(ws) == 0
    want, off = ref.verify(q, cache, table, kn, vn, tau, lens, cu, spec, 0.1, "paired", 0, 2.0 ** -11)
    close(out, want, off, "bf16")


@pytest.mark.parametrize("B", [2, 16])
def test_verify_strided_rows(B):
    """q, k and v as parts of one tensor, more rows than the batch has."""
    lens = (50, 128)
    cache, table, cu, q, kn, vn, tau = case(11, lens, [B] * 2, "paired", "bf16", 4, 2, 128)
    T = q.shape[0]
    fused = torch.randn(T + 3, 12, 128).bfloat16()
    fused[:T, :8], fused[:T, 8:10], fused[:T, 10:] = q, kn, vn
    f = fused.cuda()
    spec = dict(base=1e4)
    out = torch.full((T + 3, 8, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    out, ws = verify(f[:, :8], cache.cuda(), table, f[:, 8:10], f[:, 10:], i32(tau), lens, cu, B, spec, 0.1, "paired", out=out)
    assert pkg.read_status(ws) == 0 and (out[T:] == 7).all()
    same, _ = verify(q.cuda(), cache.cuda(), table, kn.cuda(), vn.cuda(), i32(tau), lens, cu, B, spec, 0.1, "paired")
    assert torch.equal(out[:T], same)


def test_cache_past_32_bit_offsets():
    """Pages beyond 4 GB: append, read and attention find them."""
    hd, H = 128, 8
    pages = (5 << 30) // (H * 18 * hd)
    cache = torch.zeros(pages, H, 18 * hd, dtype=torch.uint8, device="cuda")
    g = torch.Generator().manual_seed(5)
    ids = torch.tensor([[pages - 1, pages - 7, pages - 3, 2]])
    small = torch.tensor([[0, 1, 2, 3]])
    n, B = 50, 2
    k, v = (torch.randn(n, H, hd, generator=g).bfloat16().cuda() for _ in range(2))
    tiny = torch.zeros(4, H, 18 * hd, dtype=torch.uint8, device="cuda")
    spec = dict(base=1e4)
    put(k, v, [0], [n], ids, cache, spec)
    put(k, v, [0], [n], small, tiny, spec)
    assert torch.equal(cache[ids[0].cuda()], tiny)
    q, kn, vn = (torch.randn(B, h, hd, generator=g).bfloat16().cuda() for h in (32, H, H))
    for b in (B,):
        one, _ = verify(q, cache, ids, kn, vn, None, [n], cu_of([b]), b, spec, 0.1, "causal")
        two, _ = verify(q, tiny, small, kn, vn, None, [n], cu_of([b]), b, spec, 0.1, "causal")
        assert torch.equal(one, two)
    kr, vr, k2, v2 = (torch.empty(n, H, hd, device="cuda") for _ in range(4))
    pkg.kv4_read(cache, i32(ids), i32([0]), i32([0, n]), kr, vr, workspace())
    pkg.kv4_read(tiny, i32(small), i32([0]), i32([0, n]), k2, v2, workspace())
    assert torch.equal(kr, k2) and torch.equal(vr, v2)


def test_other_stream_and_captured_chain():
    """Append, attention and read-back captured on a stream of their own and replayed equal the eager calls."""
    hd, H, G, B = 128, 2, 4, 4
    g = torch.Generator().manual_seed(6)
    lens = [100, 31]
    table, total = tables(g, [8, 3])
    first = make_cache(g, total, H, hd).cuda()
    x = [torch.randn(2 * B, h, hd, generator=g).bfloat16().cuda() for h in (G * H, H, H)]
    spec = pkg.rope_spec(base=1e4)
    cache, out = first.clone(), torch.empty(2 * B, G * H, hd, dtype=torch.bfloat16, device="cuda")
    kr, vr = (torch.empty(2 * B, H, hd, device="cuda") for _ in range(2))
    t, L, cu, cur = i32(table), i32(lens), i32([0, B, 2 * B]), i32([0, B, 2 * B])
    args = (x[0], cache, t, x[1], x[2], None, L, cu, out)
    ws = workspace(pkg.kv4_verify_workspace_size(*args, 2 * B, B, spec, 0.1, order=ORDER["causal"]))

    def chain():
        pkg.kv4_verify(*args, ws, 2 * B, B, spec, 0.1, order=ORDER["causal"])
        pkg.kv4_append(x[1], x[2], L, cur, cache, t, ws, spec)
        pkg.kv4_read(cache, t, L, cur, kr, vr, ws)

    chain()
    want = [y.clone() for y in (out, cache, kr, vr)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        cache.copy_(first)
        chain()
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, b) for a, b in zip(want, (out, cache, kr, vr)))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        chain()
    for _ in range(3):
        cache.copy_(first)
        for y in (out, kr, vr):
            y.fill_(0)
        graph.replay()
        assert all(torch.equal(a, b) for a, b in zip(want, (out, cache, kr, vr)))
    assert pkg.read_status(ws) == 0


@pytest.mark.parametrize("B", [1, 2, 3, 6, 16])
@pytest.mark.parametrize("hd", [128, 64])
def test_verify_references_that_move_apart(B, hd):
    """Rows of many sizes over pages of many sizes: each row's largest score moves at blocks of its own, by little and by
    much; one row holds a NaN and one an infinity."""
    lens, g = (1500, 333, 2049), torch.Generator().manual_seed(77 + B)
    cache, table, cu, q, kn, vn, tau = case(B, lens, [B] * 3, "paired", "bf16", 4, 2, hd)
    ks = cache[..., 16 * hd:17 * hd]
    step = torch.randint(0, 6, cache.shape[:1] + (1, 1), generator=g)
    spare = ks >= 0xf8
    ks.copy_(torch.where(spare, ks, (0x50 + 8 * step + torch.randint(0, 8, ks.shape, generator=g)).to(torch.uint8)))
    q *= 2.0 ** torch.randint(-3, 3, q.shape[:2] + (1,), generator=g).to(q)
    q[1, 0, 3], q[0, 5, 7] = float("nan"), float("inf")
    out, ws = verify(q.cuda(), cache.cuda(), table, kn.cuda(), vn.cuda(), i32(tau), lens, cu, B, dict(base=1e4), 0.09, "paired")
    assert pkg.read_status(ws) == 0
    want, off = ref.verify(q, cache, table, kn, vn, tau, lens, cu, dict(base=1e4), 0.09, "paired", 0, 2.0 ** -11)
    # each of the at most 2049 + 32 products may be off by 2^-32 of its row's largest weight times the value
    v = max(float(ref.rows(cache, table, b, 0, n)[1].abs().nan_to_num(0).max()) for b, n in enumerate(lens))
    close(out, want, off + 2081 * 2.0 ** -32 * max(v, float(vn.abs().max())), "bf16")
