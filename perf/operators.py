"""The operators of a serving loop whose KV cache is held in 8 bits, and the
cases they are measured on.

Four operators, used one after another by a loop of verification passes:

``rope``    rotary positions of query and key rows: half or interleaved
            pairs, all of the head or its first part, frequencies scaled for
            long contexts; backwards (the gradient) as well.
``map``     block tables and slot maps from request lengths: pages taken from
            and given back to a ring of free pages.
``append``  keys (rotated) and values put into an e4m3 paged cache with one
            power-of-two scale for each page and head.
``verify``  attention of new tokens over that cache: SimSD's paired layout,
            draft-graph nodes, or causal tokens (one token: a decode step).

``run`` computes each in elementary torch operations, or, where ``own`` is
true, by the package's calls.
"""
import math

import torch

own = False

PAGE = 16           # tokens of a cache page
E4M3_MAX = 448.0    # largest finite e4m3 value
EXP_LO, EXP_HI = -64, 7   # range of a page's scale exponent


# --------------------------------------------------------------------- cases
def _rope_case(name, rows, dtype, style, rotary, scaling, Hq=32, Hkv=8, hd=128, fused=False,
               inverse=False, pos_max=32768):
    return dict(name=name, op="rope", rows=rows, dtype=dtype, style=style, rotary=rotary,
                scaling=scaling, Hq=Hq, Hkv=Hkv, hd=hd, fused=fused, inverse=inverse, pos_max=pos_max)


def _map_case(name, batch, lo, hi, new, fresh, ends):
    return dict(name=name, op="map", batch=batch, lo=lo, hi=hi, new=new, fresh=fresh, ends=ends)


def _append_case(name, batch, start_lo, start_hi, n_lo, n_hi, dtype, style, scaling, Hkv=8, hd=128):
    return dict(name=name, op="append", batch=batch, start_lo=start_lo, start_hi=start_hi, n_lo=n_lo,
                n_hi=n_hi, dtype=dtype, style=style, scaling=scaling, Hkv=Hkv, hd=hd)


def _verify_case(name, batch, lo, hi, b_lo, b_hi, order, dtype="bf16", Hq=32, Hkv=8, hd=128, node=0,
                 style="half", rotary=0, scaling="plain"):
    return dict(name=name, op="verify", batch=batch, lo=lo, hi=hi, b_lo=b_lo, b_hi=b_hi, order=order,
                dtype=dtype, Hq=Hq, Hkv=Hkv, hd=hd, node=node, style=style, rotary=rotary,
                scaling=scaling)


def listed():
    return [
        # the gradient of the rotation for one pass's rows of 16 sequences (2B = 8): a call that is
        # all latency; interleaved pairs over the first half of the head, as partial-rotary models do
        _rope_case("rope step 128 rows f32 back", 128, "f32", "interleaved", 64, "linear", inverse=True),
        # a long prompt's queries and keys, read where a fused projection left them
        _rope_case("rope prompt 262144 rows bf16", 262144, "bf16", "half", 0, "yarn", fused=True,
                   pos_max=131072),
        # what a serving loop does between two passes: 256 running requests, a few new tokens each,
        # some of them finished
        _map_case("map step 256", 256, 256, 8192, 16, False, 0.05),
        # 256 requests admitted at once: every page, and a slot for every prompt token
        _map_case("map prompts 256", 256, 0, 0, 8192, True, 0.0),
        # committing the accepted tokens of one pass into pages that are partly full
        _append_case("append step 64x8", 64, 1000, 4096, 1, 8, "bf16", "half", "plain"),
        # a batch of prompts going into the cache
        _append_case("append prompts 256", 256, 0, 0, 256, 8192, "bf16", "half", "banded"),
        # the smallest verification: one sequence, fp32, head dim 64
        _verify_case("verify tiny f32 1x64 B4", 1, 64, 64, 4, 4, "paired", "f32", 4, 2, 64),
        # one token for each of 64 requests: an ordinary decode step
        _verify_case("verify decode 64x<=4096", 64, 1, 4096, 1, 1, "causal"),
        # the verification step's configurations
        _verify_case("verify 16x1024 B4", 16, 1024, 1024, 4, 4, "paired"),
        _verify_case("verify 64x4096 B8", 64, 4096, 4096, 8, 8, "paired"),
        _verify_case("verify 8x32768 B16", 8, 32768, 32768, 16, 16, "paired", scaling="yarn"),
        _verify_case("verify 256x256-8192 B4-8", 256, 256, 8192, 4, 8, "paired"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "map", "append", "verify", "verify"])
    style = rng.choice(["half", "interleaved"])
    scaling = rng.choice(["plain", "linear", "ntk", "yarn", "banded"])
    if op == "rope":
        hd = rng.choice([64, 128])
        c = _rope_case("", _log(rng, 1, 200000), rng.choice(["f32", "bf16"]), style,
                       rng.choice([0, hd // 2, hd // 4, 24, 50]), scaling, rng.choice([4, 12, 32]),
                       rng.choice([1, 4, 8]), hd, rng.random() < 0.5, rng.random() < 0.5,
                       _log(rng, 64, 1 << 20))
        if c["dtype"] == "f32":
            c["rows"] = max(1, c["rows"] // 2)
    elif op == "map":
        fresh = rng.random() < 0.4
        hi = _log(rng, 16, 8192)
        c = _map_case("", _log(rng, 1, 256), 0 if fresh else max(1, hi // 16), 0 if fresh else hi,
                      hi if fresh else _log(rng, 1, 64), fresh, 0.0 if fresh else 0.1)
    elif op == "append":
        n_hi = _log(rng, 1, 8000)
        s_hi = rng.choice([0, _log(rng, 1, 4096)])
        c = _append_case("", _log(rng, 1, 128), s_hi // 3, s_hi, max(1, n_hi // 20), n_hi,
                         rng.choice(["f32", "bf16"]), style, scaling, rng.choice([1, 2, 8]),
                         rng.choice([64, 128]))
    else:
        dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
        order = rng.choice(["paired", "nodes", "causal"])
        hd = rng.choice([64, 128])
        Hkv = rng.choice([1, 2, 8])
        G = rng.choice([1, 2, 4, 7])
        hi = _log(rng, 1, 600 if dtype == "f32" else 16384)
        batch = _log(rng, 1, max(1, min(256, (4096 if dtype == "f32" else 400000) // hi)))
        node = rng.choice([2, 4, 8]) if order == "nodes" else 0
        b = rng.choice([1, 3, 8]) if dtype == "f32" else rng.choice([1, 2, 5, 8, 16, 32])
        b_lo, b_hi = (node, node * rng.choice([1, 2, 4])) if node else (max(1, b // 2), b)
        c = _verify_case("", batch, hi // 3, hi, b_lo, b_hi, order, dtype, Hkv * G, Hkv, hd, node, style,
                         rng.choice([0, 0, hd // 2]), scaling)
    del c["name"]
    return c


# -------------------------------------------------------------------- inputs
def _dtype(case):
    return torch.float32 if case["dtype"] == "f32" else torch.bfloat16


def _spec(case):
    """The rotary description of a case as keyword arguments of rope_spec."""
    d = dict(base=1.0e6, rotary_dim=case.get("rotary", 0), interleaved=case["style"] == "interleaved",
             scaling=case["scaling"])
    if case["scaling"] in ("linear", "ntk"):
        d.update(factor=4.0)
    elif case["scaling"] == "yarn":
        d.update(factor=4.0, original_len=32768, fast=32.0, slow=1.0)
    elif case["scaling"] == "banded":
        d.update(factor=8.0, original_len=8192, fast=4.0, slow=1.0)
    return d


def _ints(gen, lo, hi, n):
    return torch.randint(lo, hi + 1, (n,), generator=gen, dtype=torch.int64)


def _lengths(gen, lo, hi, n, step=1):
    """n lengths of lo..hi (multiples of step), the largest among them."""
    v = _ints(gen, lo // step, hi // step, n) * step
    v[0] = hi // step * step
    return v


def _sizes(case):
    """A case's lengths, one row for each sequence: the same for every seed, which orders them."""
    gen = torch.Generator().manual_seed(1)
    n, op = case["batch"], case["op"]
    if op == "map":
        lens = _lengths(gen, case["lo"], case["hi"], n)
        new = _lengths(gen, max(1, case["new"] // 32), case["new"], n)
        held = torch.zeros(n, dtype=torch.int64) if case["fresh"] else (lens + PAGE - 1) // PAGE
        go_on = (torch.rand(n, generator=gen) >= case["ends"]).long()   # 0: a finished request
        go_on[0] = 1
        return torch.stack([lens * go_on, new * go_on, held], 1)
    if op == "append":
        return torch.stack([_lengths(gen, case["start_lo"], case["start_hi"], n),
                            _lengths(gen, case["n_lo"], case["n_hi"], n)], 1)
    return torch.stack([_lengths(gen, case["lo"], case["hi"], n),
                        _lengths(gen, case["b_lo"], case["b_hi"], n, max(1, case["node"]))], 1)


def _cu(n):
    return torch.cat([torch.zeros(1, dtype=torch.int64), n.cumsum(0)])


def _i32(t):
    return t.to(torch.int32).cuda()


def _quantise(x):
    """[pages, heads, PAGE, hd] values -> e4m3 codes and e8m0 scales of their pages and heads."""
    m, e = torch.frexp(x.abs().amax((2, 3)))
    ex = torch.where(m > 0, e - 9 + (m > 0.875).int(), EXP_LO).clamp(EXP_LO, EXP_HI)
    y = torch.ldexp(x, -ex[:, :, None, None]).clamp(-E4M3_MAX, E4M3_MAX)
    return y.to(torch.float8_e4m3fn), (ex + 127).to(torch.uint8).view(torch.float8_e8m0fnu)


def _cache(dev_gen, pages, heads, hd):
    """A cache that holds data in every page: normal values whose size differs from head to head."""
    codes = torch.empty((pages, heads, PAGE, hd), dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
    scale = torch.empty((pages, heads), dtype=torch.uint8, device="cuda").view(torch.float8_e8m0fnu)
    size = torch.exp2(torch.rand((1, heads, 1, 1), generator=dev_gen, device="cuda") * 2 - 1)
    for p in range(0, pages, 16384):
        n = min(16384, pages - p)
        x = torch.randn((n, heads, PAGE, hd), generator=dev_gen, device="cuda") * size
        c, s = _quantise(x)
        codes[p:p + n] = c
        scale.view(torch.uint8)[p:p + n] = s.view(torch.uint8)
    return codes, scale


def _normal(dev_gen, shape, dtype, sd=1.0):
    return (torch.randn(shape, generator=dev_gen, device="cuda") * sd).to(dtype)


def _table(gen, pages):
    """Block table of sequences holding `pages` pages each, ids shuffled; 0 past a row's end."""
    n, width = int(pages.sum()), max(1, int(pages.max()))
    ids = torch.randperm(max(1, n), generator=gen)
    j = torch.arange(width)[None, :]
    idx = (_cu(pages)[:-1, None] + j).clamp(max=max(0, n - 1))
    return torch.where(j < pages[:, None], ids[idx], 0), max(1, n)


def prepare(case, seed):
    gen = torch.Generator().manual_seed(seed)
    dg = torch.Generator(device="cuda").manual_seed(seed)
    s = dict(case=dict(case))
    op = case["op"]
    if op != "rope":
        n = case["batch"]
        sizes = _sizes(case)[torch.randperm(n, generator=gen)].unbind(1)
    if op == "rope":
        T, Hq, Hkv, hd = case["rows"], case["Hq"], case["Hkv"], case["hd"]
        dt = _dtype(case)
        if case["fused"]:
            row = torch.empty((T, Hq + 2 * Hkv, hd), dtype=dt, device="cuda").normal_(generator=dg)
            s["q"], s["k"] = row[:, :Hq], row[:, Hq:Hq + Hkv]
        else:
            s["q"] = torch.empty((T, Hq, hd), dtype=dt, device="cuda").normal_(generator=dg)
            s["k"] = torch.empty((T, Hkv, hd), dtype=dt, device="cuda").normal_(generator=dg)
        s["positions"] = torch.randint(0, case["pos_max"], (T,), generator=dg, device="cuda", dtype=torch.int32)
        s["q_out"] = torch.empty((T, Hq, hd), dtype=dt, device="cuda")
        s["k_out"] = torch.empty((T, Hkv, hd), dtype=dt, device="cuda")
    elif op == "map":
        lens, new, held = sizes
        need = (lens + new + PAGE - 1) // PAGE
        width = int(torch.maximum(need, held).max()) + 1
        cap = int(held.sum() + need.sum()) + 8
        ids = torch.randperm(cap, generator=gen)
        j = torch.arange(width)[None, :]
        at = (_cu(held)[:-1, None] + j).clamp(max=cap - 1)
        s["block_table"] = _i32(torch.where(j < held[:, None], ids[at], 0))
        n_held, head = int(held.sum()), int(_ints(gen, 0, cap - 1, 1))
        ring = torch.full((cap,), -1, dtype=torch.int64)
        free = ids[n_held:]
        ring[(head + torch.arange(len(free))) % cap] = free
        s["free_pages"], s["queue"] = _i32(ring), _i32(torch.tensor([head, len(free)]))
        s["lens"], s["held"], s["cu_n"] = _i32(lens), _i32(held), _i32(_cu(new))
        s["total_n"] = int(new.sum())
        s["held_out"], s["queue_out"] = torch.empty_like(s["held"]), torch.empty_like(s["queue"])
        s["served"] = torch.empty_like(s["held"])
        s["slots"] = torch.full((max(1, s["total_n"]),), -1, dtype=torch.int64, device="cuda")
    elif op == "append":
        Hkv, hd, dt = case["Hkv"], case["hd"], _dtype(case)
        start, new = sizes
        pages = (start + new + PAGE - 1) // PAGE
        table, total = _table(gen, pages)
        s["block_table"] = _i32(table)
        s["k_cache"], s["k_scale"] = _cache(dg, total, Hkv, hd)
        s["v_cache"], s["v_scale"] = _cache(dg, total, Hkv, hd)
        s["start"], s["cu_n"] = _i32(start), _i32(_cu(new))
        s["total_n"] = int(new.sum())
        s["items"] = int(((start + new - 1) // PAGE - start // PAGE + 1).sum())
        s["k"] = _normal(dg, (s["total_n"], Hkv, hd), dt)
        s["v"] = _normal(dg, (s["total_n"], Hkv, hd), dt, 2.0)
    else:
        Hq, Hkv, hd, dt = case["Hq"], case["Hkv"], case["hd"], _dtype(case)
        lens, Bs = sizes
        per = 2 if case["order"] == "paired" else 1
        cu_B = _cu(Bs)
        T = per * int(cu_B[-1])
        table, total = _table(gen, (lens + PAGE - 1) // PAGE)
        s["block_table"] = _i32(table)
        s["k_cache"], s["k_scale"] = _cache(dg, total, Hkv, hd)
        s["v_cache"], s["v_scale"] = _cache(dg, total, Hkv, hd)
        s["tau"] = _i32(torch.cat([torch.randperm(int(b), generator=gen) + 1 for b in Bs]))
        s["lens"], s["cu_B"] = _i32(lens), _i32(cu_B)
        s["total_B"], s["B_max"], s["per"], s["L_max"] = int(cu_B[-1]), int(Bs.max()), per, int(lens.max())
        s["q"] = _normal(dg, (T, Hq, hd), dt)
        s["k_new"], s["v_new"] = _normal(dg, (T, Hkv, hd), dt), _normal(dg, (T, Hkv, hd), dt)
        s["out"] = torch.empty_like(s["q"])
        s["sm_scale"] = 1.0 / math.sqrt(hd)
    return s


# ----------------------------------------------------------------- plain form
def _freqs(case, hd):
    """Inverse frequencies (64 bits) of the rotated pairs, and the factor on cos and sin."""
    p = _spec(case)
    rd = p["rotary_dim"] or hd
    i = torch.arange(rd // 2, dtype=torch.float64, device="cuda")
    base, f = p["base"], p.get("factor", 1.0)
    inv, mul = base ** (-2.0 * i / rd), 1.0
    if p["scaling"] == "linear":
        inv = inv / f
    elif p["scaling"] == "ntk":
        inv = (base * f ** (rd / (rd - 2.0))) ** (-2.0 * i / rd)
    elif p["scaling"] == "yarn":
        at = lambda turns: rd * math.log(p["original_len"] / (2 * math.pi * turns)) / (2 * math.log(base))  # noqa: E731
        low, high = max(math.floor(at(p["fast"])), 0), min(math.ceil(at(p["slow"])), rd - 1)
        ramp = ((i - low) / max(high - low, 0.001)).clamp(0, 1)
        inv, mul = inv * (1 - ramp) + inv / f * ramp, 0.1 * math.log(f) + 1.0
    elif p["scaling"] == "banded":
        turns = p["original_len"] * inv / (2 * math.pi)
        mix = ((turns - p["slow"]) / (p["fast"] - p["slow"])).clamp(0, 1)
        inv = inv / f * (1 - mix) + inv * mix
    return inv, mul


def _rotate(case, x, positions, back=False):
    """x [T, H, hd] rotated at positions [T], in 32 bits (angles in 64)."""
    hd = x.shape[-1]
    inv, mul = _freqs(case, hd)
    rd = 2 * inv.numel()
    a = positions.double()[:, None] * inv[None, :]
    c, s = (a.cos() * mul).float()[:, None, :], (a.sin() * mul).float()[:, None, :]
    if back:
        s = -s
    x = x.float()
    y = x.clone()
    if case["style"] == "interleaved":
        u, v = x[..., 0:rd:2], x[..., 1:rd:2]
        y[..., 0:rd:2], y[..., 1:rd:2] = u * c - v * s, v * c + u * s
    else:
        u, v = x[..., :rd // 2], x[..., rd // 2:rd]
        y[..., :rd // 2], y[..., rd // 2:rd] = u * c - v * s, v * c + u * s
    return y


def _map_plain(s):
    lens, held, cu = s["lens"].long(), s["held"].long(), s["cu_n"].long()
    new = cu[1:] - cu[:-1]
    head, count = s["queue"].long().unbind()
    ring, cap = s["free_pages"].clone(), s["free_pages"].numel()
    need = (lens + new + PAGE - 1) // PAGE
    grow, drop = (need - held).clamp(min=0), (held - need).clamp(min=0)
    upto, back = grow.cumsum(0), drop.cumsum(0)
    served = (grow == 0) | (upto <= count)
    grow = torch.where(served, grow, 0)
    width = s["block_table"].shape[1]
    j = torch.arange(width, device="cuda")[None, :]
    k = j - held[:, None]                                            # index among a row's new pages
    take = (head + (upto - grow)[:, None] + k) % cap
    table = torch.where((k >= 0) & (k < grow[:, None]), ring[take].long(), s["block_table"].long())
    # pages given back go behind the last free one; places past a row's own go to a spare one
    k = j - need[:, None]
    put = torch.where((k >= 0) & (k < drop[:, None]), (head + count + (back - drop)[:, None] + k) % cap, cap)
    wide = torch.cat([ring, ring[:1]])
    wide[put] = s["block_table"]
    t = torch.arange(s["total_n"], device="cuda")
    b = torch.searchsorted(cu[1:].contiguous(), t, right=True)
    pos = lens[b] + t - cu[b]
    slots = torch.where(served[b], table[b, (pos // PAGE).clamp(max=width - 1)] * PAGE + pos % PAGE, -1)
    queue = torch.stack([(head + grow.sum()) % cap, count - grow.sum() + drop.sum()])
    return dict(block_table=table.int(), free_pages=wide[:cap], slots=slots, queue=queue.int(),
                held=torch.where(served, need, held).int(), served=served.int())


def _place(s, x, codes, scale):
    """Rows x [N, H, hd] (32 bits) into the pages of the cache they belong to."""
    start, cu, table = s["start"].long(), s["cu_n"].long(), s["block_table"].long()
    n = cu[1:] - cu[:-1]
    first = start // PAGE
    count = (start + n - 1) // PAGE - first + 1
    b = torch.repeat_interleave(torch.arange(len(n), device="cuda"), count, output_size=s["items"])
    j = first[b] + torch.arange(s["items"], device="cuda") - (count.cumsum(0) - count)[b]
    page = table[b, j]
    pos = j[:, None] * PAGE + torch.arange(PAGE, device="cuda")[None, :]
    old = (pos < start[b][:, None])[:, None, :, None]
    new = ((pos >= start[b][:, None]) & (pos < (start + n)[b][:, None]))[:, None, :, None]
    row = (cu[b][:, None] + pos - start[b][:, None]).clamp(0, x.shape[0] - 1)
    v = x[row].transpose(1, 2)                                       # [items, H, PAGE, hd]
    m, e = torch.frexp(torch.where(new, v.abs(), 0).amax((2, 3)))
    ex = torch.where(m > 0, e - 9 + (m > 0.875).int(), EXP_LO).clamp(EXP_LO, EXP_HI)
    was = scale.view(torch.uint8)[page].int() - 127
    ex = torch.where(old.any(2)[..., 0], torch.maximum(ex, was), ex)
    codes_b, scale_b = codes.view(torch.uint8), scale.view(torch.uint8)
    kept = codes_b[page]
    value = kept.view(torch.float8_e4m3fn).float()
    moved = torch.ldexp(value, (was - ex)[:, :, None, None]).to(torch.float8_e4m3fn).view(torch.uint8)
    fresh = torch.ldexp(v, -ex[:, :, None, None]).clamp(-E4M3_MAX, E4M3_MAX)
    fresh = fresh.to(torch.float8_e4m3fn).view(torch.uint8)
    codes_b[page] = torch.where(new, fresh, torch.where(old, moved, kept))
    scale_b[page] = (ex + 127).to(torch.uint8)


def _append_plain(s):
    start, cu = s["start"].long(), s["cu_n"].long()
    t = torch.arange(s["total_n"], device="cuda")
    b = torch.searchsorted(cu[1:].contiguous(), t, right=True)
    _place(s, _rotate(s["case"], s["k"], start[b] + t - cu[b]), s["k_cache"], s["k_scale"])
    _place(s, s["v"].float(), s["v_cache"], s["v_scale"])


def _verify_plain(s):
    c = s["case"]
    Hq, Hkv, hd, per, n_max = c["Hq"], c["Hkv"], c["hd"], s["per"], s["per"] * s["B_max"]
    G, lens, cu = Hq // Hkv, s["lens"].long(), s["cu_B"].long()
    batch, Bs = lens.numel(), cu[1:] - cu[:-1]
    # rows of the new tokens, padded to [batch, n_max]
    j = torch.arange(n_max, device="cuda")[None, :]
    inside = j < per * Bs[:, None]
    row = (per * cu[:-1, None] + j).clamp(max=s["q"].shape[0] - 1)
    if c["order"] == "paired":
        k = torch.where(j < Bs[:, None], j, j - Bs[:, None])
        tau = s["tau"].long()[(cu[:-1, None] + k).clamp(0, s["tau"].numel() - 1)]
        slot = j >= Bs[:, None]
        ti, tj, ri, rj = tau[:, :, None], tau[:, None, :], slot[:, :, None], slot[:, None, :]
        sees = torch.where(ri, torch.where(rj, tj >= ti, tj < ti), ~rj & (tj <= ti))
    elif c["order"] == "nodes":
        k = (j % c["node"]).expand_as(row)
        sees = ((j // c["node"])[:, :, None] == (j // c["node"])[:, None, :]).expand(batch, n_max, n_max)
    else:
        k = j.expand_as(row)
        sees = (j[:, None, :] <= j[:, :, None]).expand(batch, n_max, n_max)
    sees = sees & inside[:, None, :]
    at = (lens[:, None] + k).reshape(-1)
    q = _rotate(c, s["q"][row.reshape(-1)], at).view(batch, n_max, Hkv, G, hd).permute(0, 2, 3, 1, 4)
    kn = _rotate(c, s["k_new"][row.reshape(-1)], at).view(batch, n_max, Hkv, hd).transpose(1, 2)
    vn = s["v_new"][row.reshape(-1)].float().view(batch, n_max, Hkv, hd).transpose(1, 2)
    # the cache's values, padded to the table's width
    table = s["block_table"].long()

    def held(codes, scale):
        x = codes.view(torch.uint8)[table].view(torch.float8_e4m3fn).float()
        x *= torch.exp2(scale.view(torch.uint8)[table].float() - 127)[..., None, None]
        return x.transpose(1, 2).reshape(batch, Hkv, -1, hd)

    past = torch.arange(table.shape[1] * PAGE, device="cuda")[None, :] < lens[:, None]
    q = q.reshape(batch, Hkv, G * n_max, hd) * s["sm_scale"]
    keys = held(s["k_cache"], s["k_scale"])
    old = (q @ keys.transpose(2, 3)).masked_fill_(~past[:, None, None, :], -math.inf)
    del keys
    new = (q @ kn.transpose(2, 3)).view(batch, Hkv, G, n_max, n_max)
    new = new.masked_fill(~sees[:, None, None], -math.inf).view(batch, Hkv, G * n_max, n_max)
    top = torch.maximum(old.amax(-1), new.amax(-1))[..., None]
    top = torch.where(top == -math.inf, 0, top)
    old, new = old.sub_(top).exp_(), (new - top).exp()
    total = old.sum(-1, keepdim=True) + new.sum(-1, keepdim=True)
    o = (old @ held(s["v_cache"], s["v_scale"]) + new @ vn) / total
    o = o.view(batch, Hkv, G, n_max, hd).permute(0, 3, 1, 2, 4).reshape(batch, n_max, Hq, hd)
    s["out"][row[inside]] = o[inside].to(s["out"].dtype)


# ------------------------------------------------------------- one pass of each
def _run_own(s):
    import speculative_decoding_diffusion_gb300 as pkg
    c, op = s["case"], s["case"]["op"]
    if "spec" not in s and op != "map":
        s["spec"] = pkg.rope_spec(**_spec(c))
    if op == "rope":
        pkg.rope(s["q"], s["positions"], s["spec"], s["q_out"], s["k"], s["k_out"], inverse=c["inverse"])
        return s["q_out"], s["k_out"]
    if op == "map":
        if "ws" not in s:
            n = pkg.page_map_workspace_size(s["lens"], s["block_table"], s["free_pages"], s["total_n"])
            s["ws"] = torch.zeros(n, dtype=torch.uint8, device="cuda")
        pkg.page_map(s["lens"], s["cu_n"], s["held"], s["queue"], s["free_pages"], s["block_table"],
                     s["held_out"], s["queue_out"], s["served"], s["slots"], s["ws"], s["total_n"])
        return dict(block_table=s["block_table"], free_pages=s["free_pages"],
                    slots=s["slots"][:s["total_n"]], queue=s["queue_out"], held=s["held_out"],
                    served=s["served"])
    if op == "append":
        if "ws" not in s:
            s["ws"] = torch.zeros(256, dtype=torch.uint8, device="cuda")
        pkg.kvq_append(s["k"], s["v"], s["start"], s["cu_n"], s["k_cache"], s["v_cache"], s["k_scale"],
                       s["v_scale"], s["block_table"], s["ws"], s["spec"])
        return s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"]
    order = dict(paired=pkg.SIMSD_ORDER_PAIRED, nodes=pkg.SIMSD_ORDER_NODES, causal=pkg.SIMSD_ORDER_CAUSAL)[c["order"]]
    args = (s["q"], s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"], s["block_table"], s["k_new"],
            s["v_new"], s["tau"], s["lens"], s["cu_B"], s["out"])
    kw = dict(order=order, node_size=c["node"])
    if "ws" not in s:
        n = pkg.kvq_verify_workspace_size(*args, s["total_B"], s["B_max"], s["spec"], s["sm_scale"], **kw)
        s["ws"] = torch.zeros(n, dtype=torch.uint8, device="cuda")
    pkg.kvq_verify(*args, s["ws"], s["total_B"], s["B_max"], s["spec"], s["sm_scale"], **kw)
    return s["out"]


def run(state):
    if own:
        return _run_own(state)
    s, op = state, state["case"]["op"]
    if op == "rope":
        s["q_out"].copy_(_rotate(s["case"], s["q"], s["positions"], s["case"]["inverse"]))
        s["k_out"].copy_(_rotate(s["case"], s["k"], s["positions"], s["case"]["inverse"]))
        return s["q_out"], s["k_out"]
    if op == "map":
        return _map_plain(s)
    if op == "append":
        _append_plain(s)
        return s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"]
    _verify_plain(s)
    return s["out"]


def work(case):
    """Bytes and operations of one pass: inputs read once, outputs written once."""
    op = case["op"]
    es = 4 if case.get("dtype") == "f32" else 2
    if op == "rope":
        x = case["rows"] * (case["Hq"] + case["Hkv"]) * case["hd"]
        return dict(bytes=2 * x * es + 4 * case["rows"], flops=3 * x)
    sizes = _sizes(case)
    if op == "map":
        lens, new, held = sizes.unbind(1)
        pages = int(((lens + new + PAGE - 1) // PAGE - held).abs().sum())
        return dict(bytes=20 * case["batch"] + 8 * pages + 8 * int(new.sum()), flops=4 * int(new.sum()))
    if op == "append":
        x = int(sizes[:, 1].sum()) * case["Hkv"] * case["hd"]
        return dict(bytes=2 * x * (es + 1), flops=6 * x)
    lens, n = sizes[:, 0], sizes[:, 1] * (2 if case["order"] == "paired" else 1)
    P, T, row = int(lens.sum()), int(n.sum()), case["Hkv"] * case["hd"]
    read = 2 * P * (row + case["Hkv"] / PAGE) + 2 * T * row * es + 2 * T * case["Hq"] * case["hd"] * es
    return dict(bytes=read, flops=4 * int((lens * n + n * n).sum()) * case["Hq"] * case["hd"])


# ------------------------------------------------------ the definition, in 64 bits
def _turn(case, x, pos, sign=1.0):
    """The rotation as a product of complex numbers."""
    p = _spec(case)
    hd = x.shape[-1]
    rd = p["rotary_dim"] or hd
    f = p.get("factor", 1.0)
    freq, size = [], 1.0
    for i in range(rd // 2):
        w = math.exp(-2.0 * i / rd * math.log(p["base"]))
        if p["scaling"] == "linear":
            w /= f
        elif p["scaling"] == "ntk":
            w = math.exp(-2.0 * i / rd * (math.log(p["base"]) + rd / (rd - 2.0) * math.log(f)))
        elif p["scaling"] == "yarn":
            size = 1.0 + 0.1 * math.log(f)
            edge = [rd * math.log(p["original_len"] / (n * 2 * math.pi)) / (2 * math.log(p["base"])) for n in (p["fast"], p["slow"])]
            lo, hi = max(0, math.floor(edge[0])), min(rd - 1, math.ceil(edge[1]))
            r = min(1.0, max(0.0, (i - lo) / max(hi - lo, 0.001)))
            w = w / f * r + w * (1.0 - r)
        elif p["scaling"] == "banded":
            n = p["original_len"] / (2 * math.pi / w)
            r = 1.0 if n > p["fast"] else 0.0 if n < p["slow"] else (n - p["slow"]) / (p["fast"] - p["slow"])
            w = r * w + (1.0 - r) * w / f
        freq.append(w)
    turn = torch.polar(torch.tensor(size, dtype=torch.float64, device="cuda"),
                       sign * pos.double()[:, None] * torch.tensor(freq, dtype=torch.float64, device="cuda"))
    x = x.double()
    if case["style"] == "interleaved":
        z = torch.view_as_complex(x[..., :rd].reshape(*x.shape[:-1], rd // 2, 2).contiguous()) * turn[:, None]
        y = torch.view_as_real(z).flatten(-2)
    else:
        z = torch.complex(x[..., :rd // 2], x[..., rd // 2:rd]) * turn[:, None]
        y = torch.cat([z.real, z.imag], -1)
    return torch.cat([y, x[..., rd:]], -1)


def _code(y):
    """The e4m3 value nearest to y (|y| <= 448), ties to the even one, in 64 bits."""
    _, e = torch.frexp(y)
    step = torch.exp2((e - 4).clamp(min=-9).double())
    return torch.round(y / step) * step


def exact(case, seed):
    op = case["op"]
    if op == "map":
        return None
    s = prepare(case, seed)
    if op == "rope":
        sign = -1.0 if case["inverse"] else 1.0
        return tuple(torch.cat([_turn(case, x[i:i + 32768], s["positions"][i:i + 32768], sign)
                                for i in range(0, x.shape[0], 32768)]) for x in (s["q"], s["k"]))
    cu = s["cu_n" if op == "append" else "cu_B"].tolist()
    if op == "append":
        # page after page of sequence after sequence would be too slow for prompts: sequences one by
        # one, their pages together
        kc, vc = s["k_cache"].double(), s["v_cache"].double()
        ks, vs = s["k_scale"].double(), s["v_scale"].double()
        for b, at in enumerate(s["start"].tolist()):
            n = cu[b + 1] - cu[b]
            first, last = at // PAGE, (at + n - 1) // PAGE
            page = s["block_table"][b, first:last + 1].long()
            pos = at + torch.arange(n, device="cuda")
            k = _turn(case, s["k"][cu[b]:cu[b + 1]], pos)
            v = s["v"][cu[b]:cu[b + 1]].double()
            for x, codes, scale in ((k, kc, ks), (v, vc, vs)):
                full = torch.zeros(((last - first + 1) * PAGE, *x.shape[1:]), dtype=torch.float64, device="cuda")
                full[at - first * PAGE:at - first * PAGE + n] = x
                full = full.view(-1, PAGE, *x.shape[1:]).transpose(1, 2)
                top = full.abs().amax((2, 3))
                sc = torch.exp2((torch.ceil(torch.log2(top / E4M3_MAX)) - 1).clamp(EXP_LO, EXP_HI))
                for _ in range(2):          # the smallest power that holds top, whichever way the logarithm rounds
                    sc = torch.where(top > E4M3_MAX * sc, 2 * sc, sc).clamp(max=2.0 ** EXP_HI)
                if at % PAGE:
                    sc[0] = torch.maximum(sc[0], scale[page[0]])
                    held = codes[page[0]] * scale[page[0]][:, None, None]
                    full[0, :, :at % PAGE] = held[:, :at % PAGE]
                # _code() of a value beyond the range is not asked for: sc covers every value here
                y = _code(full / sc[:, :, None, None])
                keep = torch.zeros((last - first + 1) * PAGE, dtype=torch.bool, device="cuda")
                keep[at - first * PAGE + n:] = True
                codes[page] = torch.where(keep.view(-1, 1, PAGE, 1), codes[page], y)
                scale[page] = sc
        return kc, vc, ks, vs
    per, Hq, Hkv = s["per"], case["Hq"], case["Hkv"]
    out = torch.empty(s["out"].shape, dtype=torch.float64, device="cuda")
    for b, P in enumerate(s["lens"].tolist()):
        r = slice(per * cu[b], per * cu[b + 1])
        B = cu[b + 1] - cu[b]
        n = per * B
        i = torch.arange(n, device="cuda")
        if case["order"] == "paired":
            tau = s["tau"][cu[b]:cu[b + 1]].long()
            when = torch.cat([tau, tau])
            slot = i >= B
            off = i % B
            sees = torch.zeros((n, n), dtype=torch.bool, device="cuda")
            sees[B:, :B] = when[None, :B] < when[B:, None]
            sees[B:, B:] = when[None, B:] >= when[B:, None]
            sees[:B, :B] = when[None, :B] <= when[:B, None]
        elif case["order"] == "nodes":
            off, sees = i % case["node"], i[:, None] // case["node"] == i[None, :] // case["node"]
        else:
            off, sees = i, i[:, None] >= i[None, :]
        q, kn = _turn(case, s["q"][r], P + off), _turn(case, s["k_new"][r], P + off)
        page = s["block_table"][b, :(P + PAGE - 1) // PAGE].long()

        def all_keys(codes, scale, more):
            x = codes[page].double() * scale[page].double()[..., None, None]
            return torch.cat([x.permute(0, 2, 1, 3).reshape(-1, Hkv, case["hd"])[:P], more.double()])

        k, v = all_keys(s["k_cache"], s["k_scale"], kn), all_keys(s["v_cache"], s["v_scale"], s["v_new"][r])
        w = torch.einsum("nhgd,khd->hgnk", q.view(n, Hkv, Hq // Hkv, -1), k) * s["sm_scale"]
        w[..., P:].masked_fill_(~sees, -math.inf)
        w = torch.softmax(w, -1)
        out[r] = torch.einsum("hgnk,khd->nhgd", w, v).reshape(n, Hq, -1)
    return out
