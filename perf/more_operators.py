"""The operators of a serving loop whose KV cache is held in 4 bits, and of the
answer that it gives for its tokens; the cases they are measured on.

``append``    keys (rotated) and values quantised as they are written into
              pages of 4-bit codes with a scale for every 16 elements, and the
              pages' tokens read back (as a prompt that goes in by pieces does).
``read``      the tokens of each sequence read back from the pages.
``verify``    attention of new tokens over that cache: SimSD's paired layout,
              draft-graph nodes, or causal tokens (one token: a decode step).
``logprobs``  log probabilities of given tokens, their ranks, the entropy and
              the likeliest tokens of every row of logits.

``run`` computes each in elementary torch operations, or, where ``own`` is
true, by the package's calls.

A page and head of the cache is a record of 18 hd bytes: key codes [16][hd / 2]
(two neighbouring elements a byte, the first one low), value codes
[hd / 32][8][32] (two neighbouring tokens of an element a byte, the first one
low), key scales [16][hd / 16], value scales [8][hd / 16][2].  A code is an
e2m1 number; a scale is bits 14..7 of an fp16 number.
"""
import math

import torch

own = False

PAGE = 16              # tokens of a cache page
GROUP = 16             # elements of a scale
CODES = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]
SCALE_MAX = 10240.0    # largest scale (times 6: inside fp16)
E4M3_MAX = 448.0


# --------------------------------------------------------------------- cases
def _append_case(name, batch, start_lo, start_hi, n_lo, n_hi, dtype, style, scaling, Hkv=8, hd=128):
    return dict(name=name, op="append", batch=batch, start_lo=start_lo, start_hi=start_hi, n_lo=n_lo,
                n_hi=n_hi, dtype=dtype, style=style, scaling=scaling, Hkv=Hkv, hd=hd)


def _read_case(name, batch, start_lo, start_hi, n_lo, n_hi, dtype, Hkv=8, hd=128):
    return dict(name=name, op="read", batch=batch, start_lo=start_lo, start_hi=start_hi, n_lo=n_lo,
                n_hi=n_hi, dtype=dtype, Hkv=Hkv, hd=hd)


def _verify_case(name, batch, lo, hi, b_lo, b_hi, order, dtype="bf16", Hq=32, Hkv=8, hd=128, node=0,
                 style="half", rotary=0, scaling="plain"):
    return dict(name=name, op="verify", batch=batch, lo=lo, hi=hi, b_lo=b_lo, b_hi=b_hi, order=order,
                dtype=dtype, Hq=Hq, Hkv=Hkv, hd=hd, node=node, style=style, rotary=rotary, scaling=scaling)


def _logprobs_case(name, rows, vocab, top, dtype="bf16", temperature=1.0, pad=0):
    return dict(name=name, op="logprobs", rows=rows, vocab=vocab, top=top, dtype=dtype,
                temperature=temperature, pad=pad)


def listed():
    return [
        # committing the accepted tokens of one pass into pages that are partly full
        _append_case("append step 64x8", 64, 1000, 4096, 1, 8, "bf16", "half", "plain"),
        # a batch of prompts going into the cache
        _append_case("append prompts 128", 128, 0, 0, 256, 8192, "bf16", "half", "banded"),
        # a few short prefixes at odd places, for a check in 32 bits
        _read_case("read tiny f32 5x<=100", 5, 3, 37, 1, 100, "f32", 2, 64),
        # whole prefixes handed to another program
        _read_case("read 8x32768", 8, 0, 0, 32768, 32768, "bf16"),
        # the smallest verification: one sequence, fp32, head dim 64
        _verify_case("verify tiny f32 1x64 B4", 1, 64, 64, 4, 4, "paired", "f32", 4, 2, 64),
        # one token for each of 64 requests: an ordinary decode step
        _verify_case("verify decode 64x<=4096", 64, 1, 4096, 1, 1, "causal"),
        # the verification step's configurations
        _verify_case("verify 16x1024 B4", 16, 1024, 1024, 4, 4, "paired"),
        _verify_case("verify 64x4096 B8", 64, 4096, 4096, 8, 8, "paired"),
        _verify_case("verify 8x32768 B16", 8, 32768, 32768, 16, 16, "paired", scaling="yarn"),
        _verify_case("verify 256x256-8192 B4-8", 256, 256, 8192, 4, 8, "paired"),
        # the tokens that one request commits in a pass
        _logprobs_case("logprobs 4 rows", 4, 151936, 5, "bf16", 0.7),
        # every slot of 256 requests, with 20 alternatives
        _logprobs_case("logprobs 1536 rows", 1536, 151936, 20),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "read", "verify", "verify", "verify", "logprobs"])
    style = rng.choice(["half", "interleaved"])
    scaling = rng.choice(["plain", "linear", "ntk", "yarn", "banded"])
    hd = rng.choice([64, 128])
    if op in ("append", "read"):
        n_hi = _log(rng, 1, 8000)
        s_hi = rng.choice([0, _log(rng, 1, 4096)])
        sizes = (_log(rng, 1, 64), s_hi // 3, s_hi, max(1, n_hi // 20), n_hi)
        Hkv = rng.choice([1, 2, 8])
        if op == "append":
            c = _append_case("", *sizes, rng.choice(["f32", "bf16"]), style, scaling, Hkv, hd)
        else:
            c = _read_case("", *sizes, rng.choice(["f32", "bf16", "e4m3"]), Hkv, hd)
    elif op == "logprobs":
        vocab = rng.choice([512, 32003, 50257, 151936, _log(rng, 64, 200000)])
        c = _logprobs_case("", _log(rng, 1, max(2, min(4096, 200_000_000 // vocab))), vocab,
                           rng.choice([0, 1, 5, 20, 32]), rng.choice(["f32", "bf16"]),
                           rng.choice([1.0, 0.6, 1.3]), rng.choice([0, 0, 3, 64]))
    else:
        dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
        order = rng.choice(["paired", "nodes", "causal"])
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
_TYPES = dict(f32=torch.float32, bf16=torch.bfloat16, e4m3=torch.float8_e4m3fn)


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


def _lengths(gen, lo, hi, n, step=1):
    """n lengths of lo..hi (multiples of step), the largest among them."""
    v = torch.randint(lo // step, hi // step + 1, (n,), generator=gen, dtype=torch.int64) * step
    v[0] = hi // step * step
    return v


def _sizes(case):
    """A case's lengths, one row for each sequence: the same for every seed, which orders them."""
    gen = torch.Generator().manual_seed(1)
    n = case["batch"]
    if case["op"] == "verify":
        return torch.stack([_lengths(gen, case["lo"], case["hi"], n),
                            _lengths(gen, case["b_lo"], case["b_hi"], n, max(1, case["node"]))], 1)
    return torch.stack([_lengths(gen, case["start_lo"], case["start_hi"], n),
                        _lengths(gen, case["n_lo"], case["n_hi"], n)], 1)


def _cu(n):
    return torch.cat([torch.zeros(1, dtype=torch.int64), n.cumsum(0)])


def _i32(t):
    return t.to(torch.int32).cuda()


def _normal(dev_gen, shape, dtype, sd=1.0):
    return (torch.randn(shape, generator=dev_gen, device="cuda") * sd).to(dtype)


def _table(gen, pages):
    """Block table of sequences holding `pages` pages each, ids shuffled; 0 past a row's end."""
    n, width = int(pages.sum()), max(1, int(pages.max()))
    ids = torch.randperm(max(1, n), generator=gen)
    j = torch.arange(width)[None, :]
    idx = (_cu(pages)[:-1, None] + j).clamp(max=max(0, n - 1))
    return torch.where(j < pages[:, None], ids[idx], 0), max(1, n)


def _quantise(x):
    """[.., hd] values in 32 bits -> codes 0..15 and scale bytes [.., hd / 16]."""
    g = x.unflatten(-1, (-1, GROUP))
    top = g.abs().amax(-1)
    # (divided by a tensor: by a number it is a product with a rounded 1 / 6)
    want = (top / torch.full_like(top, 6.0)).double()
    _, e = torch.frexp(want)
    step = torch.exp2((e - 4).clamp(min=-17).double())
    scale = (torch.round(want / step) * step).clamp(max=SCALE_MAX).to(torch.float16)
    y = (g.abs() / scale.float()[..., None]).nan_to_num_(0.0, posinf=6.0)
    # borders between neighbours; one in the middle goes to the even code
    code = ((y > 0.25).byte() + (y >= 0.75).byte() + (y > 1.25).byte() + (y >= 1.75).byte() +
            (y > 2.5).byte() + (y >= 3.5).byte() + (y > 5).byte())
    code = torch.where(g < 0, code + 8, code)
    code = torch.where((scale == 0)[..., None], 0, code)
    return code.flatten(-2), (scale.view(torch.int16) >> 7).byte()


def _pack(kc, ks, vc, vs):
    """Codes [N, H, 16, hd] and scale bytes [N, H, 16, hd / 16] of keys and values -> records."""
    n, h, _, hd = kc.shape
    k = kc[..., 0::2] | kc[..., 1::2] << 4
    v = (vc[:, :, 0::2] | vc[:, :, 1::2] << 4).view(n, h, 8, hd // 32, 32).transpose(2, 3)
    s = vs.view(n, h, 8, 2, hd // GROUP).transpose(3, 4)
    return torch.cat([x.flatten(2) for x in (k, v, ks, s)], 2)


def _unpack(rec):
    """Records [N, H, 18 hd] -> what _pack took."""
    n, h, size = rec.shape
    hd = size // 18
    k = rec[..., :8 * hd].view(n, h, PAGE, hd // 2)
    v = rec[..., 8 * hd:16 * hd].view(n, h, hd // 32, 8, 32).transpose(2, 3).reshape(n, h, 8, hd)
    ks = rec[..., 16 * hd:17 * hd].view(n, h, PAGE, hd // GROUP)
    vs = rec[..., 17 * hd:].view(n, h, 8, hd // GROUP, 2).transpose(3, 4).reshape(n, h, PAGE, hd // GROUP)
    kc = torch.stack([k & 15, k >> 4], -1).flatten(3)
    vc = torch.stack([v & 15, v >> 4], 3).flatten(2, 3)
    return kc, ks, vc, vs


def _values(code, byte):
    """Codes [.., hd] and scale bytes [.., hd / 16] -> values in 32 bits."""
    table = torch.tensor(CODES + [-c for c in CODES], device=code.device)
    scale = (byte.to(torch.int16) << 7).view(torch.float16).float()
    return (table[code.long()].unflatten(-1, (-1, GROUP)) * scale[..., None]).flatten(-2)


def _cache(dev_gen, pages, heads, hd):
    """A cache that holds data in every page: normal values whose size differs from head to head."""
    rec = torch.empty((pages, heads, 18 * hd), dtype=torch.uint8, device="cuda")
    size = torch.exp2(torch.rand((1, heads, 1, 1), generator=dev_gen, device="cuda") * 2 - 1)
    for p in range(0, pages, 8192):
        shape = (min(8192, pages - p), heads, PAGE, hd)
        parts = [_quantise(torch.randn(shape, generator=dev_gen, device="cuda") * size) for _ in range(2)]
        rec[p:p + shape[0]] = _pack(*parts[0], *parts[1])
    return rec


def prepare(case, seed):
    gen = torch.Generator().manual_seed(seed)
    dg = torch.Generator(device="cuda").manual_seed(seed)
    s = dict(case=dict(case))
    op, dt = case["op"], _TYPES[case["dtype"]]
    if op == "logprobs":
        rows, vocab, top = case["rows"], case["vocab"], case["top"]
        x = torch.empty((rows, vocab + case["pad"]), dtype=dt, device="cuda")
        for r in range(0, rows, 256):          # normal logits, and tokens drawn from them
            y = torch.randn((min(256, rows - r), vocab + case["pad"]), generator=dg, device="cuda") * 3
            x[r:r + 256] = y.to(dt)
        s["logits"] = x[:, :vocab]
        pick = torch.empty((rows,), dtype=torch.int64, device="cuda")
        for r in range(0, rows, 256):
            y = s["logits"][r:r + 256].float() / case["temperature"]
            u = torch.rand(y.shape, generator=dg, device="cuda").clamp_(min=1e-30)
            pick[r:r + 256] = (y - (-u.log()).log()).argmax(-1)
        s["tokens"] = pick.int()
        s["logprob"], s["entropy"] = (torch.empty(rows, device="cuda") for _ in range(2))
        s["rank"] = torch.empty(rows, dtype=torch.int32, device="cuda")
        s["top_ids"] = torch.empty((rows, top), dtype=torch.int32, device="cuda") if top else None
        s["top_logprobs"] = torch.empty((rows, top), device="cuda") if top else None
        return s
    n, Hkv, hd = case["batch"], case["Hkv"], case["hd"]
    sizes = _sizes(case)[torch.randperm(n, generator=gen)].unbind(1)
    if op == "verify":
        Hq = case["Hq"]
        lens, Bs = sizes
        per = 2 if case["order"] == "paired" else 1
        cu_B = _cu(Bs)
        T = per * int(cu_B[-1])
        table, total = _table(gen, (lens + PAGE - 1) // PAGE)
        s["block_table"], s["cache"] = _i32(table), _cache(dg, total, Hkv, hd)
        s["tau"] = _i32(torch.cat([torch.randperm(int(b), generator=gen) + 1 for b in Bs]))
        s["lens"], s["cu_B"] = _i32(lens), _i32(cu_B)
        s["total_B"], s["B_max"], s["per"] = int(cu_B[-1]), int(Bs.max()), per
        s["q"] = _normal(dg, (T, Hq, hd), dt)
        s["k_new"], s["v_new"] = _normal(dg, (T, Hkv, hd), dt), _normal(dg, (T, Hkv, hd), dt)
        s["out"] = torch.empty_like(s["q"])
        s["sm_scale"] = 1.0 / math.sqrt(hd)
        return s
    start, new = sizes
    table, total = _table(gen, (start + new + PAGE - 1) // PAGE)
    s["block_table"], s["cache"] = _i32(table), _cache(dg, total, Hkv, hd)
    if op == "append":
        s["start"], s["cu_n"], s["total_n"] = _i32(start), _i32(_cu(new)), int(new.sum())
        s["items"] = int(((start + new - 1) // PAGE - start // PAGE + 1).sum())
        s["k"] = _normal(dg, (s["total_n"], Hkv, hd), dt)
        s["v"] = _normal(dg, (s["total_n"], Hkv, hd), dt, 2.0)
        # read back: from the first slot of the first page written, so older neighbours too
        new, start, dt = new + start % PAGE, start // PAGE * PAGE, torch.float8_e4m3fn
    s["from"], s["cu_read"], s["rows"] = _i32(start), _i32(_cu(new)), int(new.sum())
    s["read_items"] = int(((start + new - 1) // PAGE - start // PAGE + 1).sum())
    s["k_out"], s["v_out"] = (torch.empty((s["rows"], Hkv, hd), dtype=dt, device="cuda") for _ in range(2))
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


def _rotate(case, x, positions):
    """x [T, H, hd] rotated at positions [T], in 32 bits (angles in 64)."""
    hd = x.shape[-1]
    inv, mul = _freqs(case, hd)
    rd = 2 * inv.numel()
    a = positions.double()[:, None] * inv[None, :]
    c, s = (a.cos() * mul).float()[:, None, :], (a.sin() * mul).float()[:, None, :]
    x = x.float()
    y = x.clone()
    if case["style"] == "interleaved":
        u, v = x[..., 0:rd:2], x[..., 1:rd:2]
        y[..., 0:rd:2], y[..., 1:rd:2] = u * c - v * s, v * c + u * s
    else:
        u, v = x[..., :rd // 2], x[..., rd // 2:rd]
        y[..., :rd // 2], y[..., rd // 2:rd] = u * c - v * s, v * c + u * s
    return y


def _items(start, cu, table, items):
    """The pages that hold positions start.. of each sequence: (sequence, page id, positions [items, 16])."""
    n = cu[1:] - cu[:-1]
    first = start // PAGE
    count = torch.where(n > 0, (start + n - 1) // PAGE - first + 1, 0)
    b = torch.repeat_interleave(torch.arange(len(n), device="cuda"), count, output_size=items)
    j = first[b] + torch.arange(items, device="cuda") - (count.cumsum(0) - count)[b]
    return b, table[b, j], j[:, None] * PAGE + torch.arange(PAGE, device="cuda")[None, :]


def _append_plain(s):
    start, cu = s["start"].long(), s["cu_n"].long()
    t = torch.arange(s["total_n"], device="cuda")
    seq = torch.searchsorted(cu[1:].contiguous(), t, right=True)
    b, page, pos = _items(start, cu, s["block_table"].long(), s["items"])
    i = pos - start[b][:, None]
    new = ((i >= 0) & (i < (cu[1:] - cu[:-1])[b][:, None]))[:, None, :, None]
    row = (cu[b][:, None] + i).clamp(0, s["total_n"] - 1)
    k = _quantise(_rotate(s["case"], s["k"], start[seq] + t - cu[seq]))
    v = _quantise(s["v"].float())
    fresh = [x[row].transpose(1, 2) for x in (*k, *v)]
    s["cache"][page] = _pack(*(torch.where(new, x, old) for x, old in zip(fresh, _unpack(s["cache"][page]))))


def _read_plain(s):
    start, cu = s["from"].long(), s["cu_read"].long()
    b, page, pos = _items(start, cu, s["block_table"].long(), s["read_items"])
    i = pos - start[b][:, None]
    there = (i >= 0) & (i < (cu[1:] - cu[:-1])[b][:, None])
    row = (cu[b][:, None] + i)[there]
    kc, ks, vc, vs = _unpack(s["cache"][page])
    for out, code, byte in ((s["k_out"], kc, ks), (s["v_out"], vc, vs)):
        x = _values(code, byte).transpose(1, 2)[there]
        if out.dtype == torch.float8_e4m3fn:
            out.view(torch.uint8)[row] = x.clamp(-E4M3_MAX, E4M3_MAX).to(out.dtype).view(torch.uint8)
        else:
            out[row] = x.to(out.dtype)


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
    kc, ks, vc, vs = _unpack(s["cache"])

    def held(code, byte):
        x = _values(code, byte).to(torch.float16)       # exact: at most six significant bits
        return x[table].transpose(1, 2).reshape(batch, Hkv, -1, hd).float()

    past = torch.arange(table.shape[1] * PAGE, device="cuda")[None, :] < lens[:, None]
    q = q.reshape(batch, Hkv, G * n_max, hd) * s["sm_scale"]
    old = (q @ held(kc, ks).transpose(2, 3)).masked_fill_(~past[:, None, None, :], -math.inf)
    new = (q @ kn.transpose(2, 3)).view(batch, Hkv, G, n_max, n_max)
    new = new.masked_fill(~sees[:, None, None], -math.inf).view(batch, Hkv, G * n_max, n_max)
    top = torch.maximum(old.amax(-1), new.amax(-1))[..., None]
    top = torch.where(top == -math.inf, 0, top)
    old, new = old.sub_(top).exp_(), (new - top).exp()
    total = old.sum(-1, keepdim=True) + new.sum(-1, keepdim=True)
    o = (old @ held(vc, vs) + new @ vn) / total
    o = o.view(batch, Hkv, G, n_max, hd).permute(0, 3, 1, 2, 4).reshape(batch, n_max, Hq, hd)
    s["out"][row[inside]] = o[inside].to(s["out"].dtype)


def _logprobs_plain(s):
    c = s["case"]
    raw = s["logits"].float()
    t = s["tokens"].long()[:, None]
    x = raw - raw.amax(-1, keepdim=True)
    x = x / c["temperature"]
    e = x.exp()
    total = e.sum(-1)
    log_total = total.log()
    d = dict(logprob=x.gather(1, t)[:, 0] - log_total, entropy=log_total - (e * x).sum(-1) / total)
    del e
    mine = raw.gather(1, t)
    ahead = (raw > mine) | ((raw == mine) & (torch.arange(raw.shape[1], device="cuda")[None, :] < t))
    d["rank"] = ahead.sum(-1).int()
    if c["top"]:
        # one whole number for each (value, index): larger values first, then lower indices
        bits = (raw + 0.0).view(torch.int32).long()
        order = torch.where(bits < 0, -(bits & 0x7fffffff), bits)
        key = order * (1 << 22) + ((1 << 22) - 1 - torch.arange(raw.shape[1], device="cuda"))[None, :]
        key = torch.topk(key, c["top"], dim=-1).values
        ids = (1 << 22) - 1 - (key & ((1 << 22) - 1))
        d["top_ids"] = ids.int()
        d["top_logprobs"] = x.gather(1, ids) - log_total[:, None]
    return d


# ------------------------------------------------------------- one pass of each
def _workspace(s, size):
    if "ws" not in s:
        s["ws"] = torch.zeros(size, dtype=torch.uint8, device="cuda")
    return s["ws"]


def _run_own(s):
    import speculative_decoding_diffusion_gb300 as pkg
    c, op = s["case"], s["case"]["op"]
    if op == "logprobs":
        args = (s["logits"], s["tokens"], s["logprob"], s["rank"], s["entropy"], s["top_ids"], s["top_logprobs"])
        if "ws" not in s:
            _workspace(s, pkg.token_logprobs_workspace_size(*args))
        pkg.token_logprobs(*args, s["ws"], temperature=c["temperature"])
        d = dict(logprob=s["logprob"], entropy=s["entropy"], rank=s["rank"])
        if c["top"]:
            d.update(top_ids=s["top_ids"], top_logprobs=s["top_logprobs"])
        return d
    if op in ("append", "read"):
        ws = _workspace(s, 256)
        if op == "append":
            if "spec" not in s:
                s["spec"] = pkg.rope_spec(**_spec(c))
            pkg.kv4_append(s["k"], s["v"], s["start"], s["cu_n"], s["cache"], s["block_table"], ws, s["spec"])
        pkg.kv4_read(s["cache"], s["block_table"], s["from"], s["cu_read"], s["k_out"], s["v_out"], ws)
        return s["k_out"], s["v_out"]
    if "spec" not in s:
        s["spec"] = pkg.rope_spec(**_spec(c))
    order = dict(paired=pkg.SIMSD_ORDER_PAIRED, nodes=pkg.SIMSD_ORDER_NODES, causal=pkg.SIMSD_ORDER_CAUSAL)[c["order"]]
    args = (s["q"], s["cache"], s["block_table"], s["k_new"], s["v_new"], s["tau"], s["lens"], s["cu_B"], s["out"])
    kw = dict(order=order, node_size=c["node"])
    if "ws" not in s:
        _workspace(s, pkg.kv4_verify_workspace_size(*args, s["total_B"], s["B_max"], s["spec"], s["sm_scale"], **kw))
    pkg.kv4_verify(*args, s["ws"], s["total_B"], s["B_max"], s["spec"], s["sm_scale"], **kw)
    return s["out"]


def run(state):
    if own:
        return _run_own(state)
    s, op = state, state["case"]["op"]
    if op == "logprobs":
        return _logprobs_plain(s)
    if op == "verify":
        _verify_plain(s)
        return s["out"]
    if op == "append":
        _append_plain(s)
    _read_plain(s)
    return s["k_out"], s["v_out"]


def work(case):
    """Bytes and operations of one pass: inputs read once, outputs written once."""
    op = case["op"]
    es = dict(f32=4, bf16=2, e4m3=1)[case["dtype"]]
    if op == "logprobs":
        n = case["rows"] * case["vocab"]
        return dict(bytes=n * es + case["rows"] * (16 + 8 * case["top"]), flops=6 * n)
    sizes = _sizes(case)
    row = case["Hkv"] * case["hd"]
    held = 9 / 16                                # bytes of an element in the cache
    if op == "verify":
        lens, n = sizes[:, 0], sizes[:, 1] * (2 if case["order"] == "paired" else 1)
        P, T = int(lens.sum()), int(n.sum())
        read = 2 * P * row * held + 2 * T * row * es + 2 * T * case["Hq"] * case["hd"] * es
        return dict(bytes=read, flops=4 * int((lens * n + n * n).sum()) * case["Hq"] * case["hd"])
    n = int(sizes[:, 1].sum()) * row
    if op == "append":                           # rows in, codes out; codes in, rows of e4m3 out
        back = n + int((sizes[:, 0] % PAGE).sum()) * row
        return dict(bytes=2 * n * (es + held) + 2 * back * (held + 1), flops=10 * n)
    return dict(bytes=2 * n * (held + es), flops=2 * n)


# ------------------------------------------------------ the definition, in 64 bits
def _turn(case, x, pos):
    """The rotation as a product of complex numbers."""
    p = _spec(case)
    rd = p["rotary_dim"] or x.shape[-1]
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
                       pos.double()[:, None] * torch.tensor(freq, dtype=torch.float64, device="cuda"))
    x = x.double()
    if case["style"] == "interleaved":
        z = torch.view_as_complex(x[..., :rd].reshape(*x.shape[:-1], rd // 2, 2).contiguous()) * turn[:, None]
        y = torch.view_as_real(z).flatten(-2)
    else:
        z = torch.complex(x[..., :rd // 2], x[..., rd // 2:rd]) * turn[:, None]
        y = torch.cat([z.real, z.imag], -1)
    return torch.cat([y, x[..., rd:]], -1)


def _grid(y, least, digits):
    """y rounded to `digits` significant bits, ties to even, steps at least `least`."""
    _, e = torch.frexp(y)
    step = torch.exp2((e - digits).double()).clamp(min=least)
    return torch.round(y / step) * step


def _held(x):
    """What the cache holds for rows x [n, H, hd] in 64 bits."""
    g = x.view(*x.shape[:-1], -1, GROUP)
    top = g.abs().amax(-1, keepdim=True)
    scale = _grid(top / torch.full_like(top, 6.0), 2.0 ** -17, 4).clamp(max=SCALE_MAX)
    code = _grid(torch.where(scale > 0, g / scale, 0.0).clamp(-6, 6), 0.5, 2)
    return (code * scale).view(x.shape)


def _page_values(page):
    """Records [m, H, 18 hd] -> keys and values [16 m, H, hd], byte by byte as the format says."""
    m, H, size = page.shape
    hd = size // 18
    d = torch.arange(hd, device="cuda")
    i = torch.arange(PAGE, device="cuda")[:, None]
    at_k, odd_k = i * (hd // 2) + d // 2, (d % 2).expand(PAGE, hd)
    at_v, odd_v = 8 * hd + (d // 32) * 256 + (i // 2) * 32 + d % 32, (i % 2).expand(PAGE, hd)
    sc_k = 16 * hd + i * (hd // 16) + d // 16
    sc_v = 17 * hd + (i // 2) * (hd // 8) + d // 16 * 2 + i % 2
    out = []
    for at, odd, sc in ((at_k, odd_k, sc_k), (at_v, odd_v, sc_v)):
        code = (page[:, :, at].int() >> (4 * odd)) & 15
        ex, man = (code >> 1) & 3, (code & 1).double()
        size_of = torch.where(ex == 0, man / 2, torch.exp2(ex.double() - 1) * (1 + man / 2))
        byte = page[:, :, sc].int()
        se, sm = byte >> 3, (byte & 7).double()
        scale = torch.where(se == 0, sm * 2.0 ** -17, torch.exp2(se.double() - 15) * (1 + sm / 8))
        x = torch.where(code >= 8, -size_of, size_of) * scale
        out.append(x.transpose(1, 2).reshape(m * PAGE, H, hd))
    return out


def exact(case, seed):
    op = case["op"]
    s = prepare(case, seed)
    if op == "logprobs":
        d = dict(logprob=[], entropy=[])
        tops = []
        for r in range(0, case["rows"], 64):
            x = s["logits"][r:r + 64].double() / case["temperature"]
            p = torch.softmax(x, -1)
            lp = x - torch.logsumexp(x, -1, keepdim=True)
            d["logprob"].append(lp.gather(1, s["tokens"][r:r + 64].long()[:, None])[:, 0])
            d["entropy"].append(-(p * lp).sum(-1))
            tops.append(torch.sort(lp, descending=True).values[:, :case["top"]])
        d = {k: torch.cat(v) for k, v in d.items()}
        d["rank"] = None
        if case["top"]:
            d.update(top_ids=None, top_logprobs=torch.cat(tops))
        return d
    if op in ("append", "read"):
        cu, back = s["cu_read"].tolist(), [[], []]
        new = s["cu_n"].tolist() if op == "append" else None
        for b, at in enumerate(s["from"].tolist()):
            n = cu[b + 1] - cu[b]
            first, last = at // PAGE, (at + n - 1) // PAGE
            rows = [x[at - first * PAGE:][:n] for x in _page_values(s["cache"][s["block_table"][b, first:last + 1].long()])]
            if op == "append":
                r = slice(new[b], new[b + 1])
                pos = int(s["start"][b]) + torch.arange(new[b + 1] - new[b], device="cuda")
                rows[0][pos - at] = _held(_turn(case, s["k"][r], pos))
                rows[1][pos - at] = _held(s["v"][r].double())
                rows = [_grid(x.clamp(-E4M3_MAX, E4M3_MAX), 2.0 ** -9, 4) for x in rows]
            elif case["dtype"] == "e4m3":
                rows = [_grid(x.clamp(-E4M3_MAX, E4M3_MAX), 2.0 ** -9, 4) for x in rows]
            back[0].append(rows[0])
            back[1].append(rows[1])
        return torch.cat(back[0]), torch.cat(back[1])
    cu, per, Hq, Hkv = s["cu_B"].tolist(), s["per"], case["Hq"], case["Hkv"]
    out = torch.empty(s["out"].shape, dtype=torch.float64, device="cuda")
    for b, P in enumerate(s["lens"].tolist()):
        r = slice(per * cu[b], per * cu[b + 1])
        B = cu[b + 1] - cu[b]
        n = per * B
        i = torch.arange(n, device="cuda")
        if case["order"] == "paired":
            tau = s["tau"][cu[b]:cu[b + 1]].long()
            off = i % B
            sees = torch.zeros((n, n), dtype=torch.bool, device="cuda")
            sees[B:, :B] = tau[None, :] < tau[:, None]
            sees[B:, B:] = tau[None, :] >= tau[:, None]
            sees[:B, :B] = tau[None, :] <= tau[:, None]
        elif case["order"] == "nodes":
            off, sees = i % case["node"], i[:, None] // case["node"] == i[None, :] // case["node"]
        else:
            off, sees = i, i[:, None] >= i[None, :]
        q, kn = _turn(case, s["q"][r], P + off), _turn(case, s["k_new"][r], P + off)
        k, v = _page_values(s["cache"][s["block_table"][b, :(P + PAGE - 1) // PAGE].long()])
        k, v = torch.cat([k[:P], kn]), torch.cat([v[:P], s["v_new"][r].double()])
        w = torch.einsum("nhgd,khd->hgnk", q.view(n, Hkv, Hq // Hkv, -1), k) * s["sm_scale"]
        w[..., P:].masked_fill_(~sees, -math.inf)
        w = torch.softmax(w, -1)
        out[r] = torch.einsum("hgnk,khd->nhgd", w, v).reshape(n, Hq, -1)
    return out
