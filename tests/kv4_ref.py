"""Plain 64-bit forms of the 4-bit-cache operators for their tests, on the CPU,
from the header's definitions: the record of a page and head, the quantisation,
the append, the read-back and the attention."""
import math

import torch

import kvq_ref

PAGE, GROUP = 16, 16
F64 = torch.float64
CODES = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=F64)
NAN_BYTE = 0xfc


def scale_values(byte):
    """uint8 scale bytes -> float64 (inf and NaN from 0xf8 on)."""
    e, m = (byte.int() >> 3), (byte.int() & 7).to(F64)
    v = torch.where(e == 0, m * 2.0 ** -17, torch.exp2(e.to(F64) - 15) * (1 + m / 8))
    v = torch.where(byte.int() == 0xf8, math.inf, v)
    return torch.where(byte.int() > 0xf8, math.nan, v)


SCALES = scale_values(torch.arange(0xe3, dtype=torch.uint8))      # up to 10240


def nearest(x, values):
    """Index of the value (ascending, from 0) nearest to x >= 0, ties to the even index; exact for x of 32 bits."""
    mid = (values[1:] + values[:-1]) / 2
    i = torch.searchsorted(mid, x.contiguous())                    # mid[i - 1] < x <= mid[i]
    tie = (i < len(mid)) & (x == mid[i.clamp(max=len(mid) - 1)])
    return torch.where(tie & (i % 2 == 1), i + 1, i)


def scale_bytes(x):
    """x [.., hd] -> bytes [.., hd / 16]."""
    top = x.unflatten(-1, (-1, GROUP)).abs().amax(-1)
    odd = ~torch.isfinite(x.unflatten(-1, (-1, GROUP))).all(-1)
    i = nearest(torch.where(odd, 0.0, top), SCALES * 6)            # (6 * a middle between scales is exact)
    return torch.where(odd, NAN_BYTE, i).to(torch.uint8)


def codes(x, byte):
    """x [.., hd] for scale bytes [.., hd / 16] -> codes 0..15."""
    s = scale_values(byte)[..., None]
    g = x.unflatten(-1, (-1, GROUP))
    mid = (CODES[1:] + CODES[:-1]) / 2
    n = torch.zeros(g.shape, dtype=torch.int64)
    for i, m in enumerate(mid):                                    # m * s is exact
        n += ((g.abs() > m * s) if i % 2 == 0 else (g.abs() >= m * s)).long()
    n = torch.where(s == 0, 0, n)
    return (n + 8 * (g < 0)).flatten(-2).to(torch.uint8)


def values(code, byte):
    v = CODES[(code & 7).long()] * torch.where(code >= 8, -1.0, 1.0).to(F64)
    return (v.unflatten(-1, (-1, GROUP)) * scale_values(byte)[..., None]).flatten(-2)


def places(hd):
    """Where element d of token i lies: byte index and shift of its key and value codes, byte index of their scales."""
    i, d = torch.arange(PAGE)[:, None], torch.arange(hd)[None, :]
    return ((i * hd // 2 + d // 2, (4 * (d % 2)).expand(PAGE, hd), 16 * hd + i * hd // 16 + d // 16),
            (8 * hd + (d // 32) * 256 + (i // 2) * 32 + d % 32, (4 * (i % 2)).expand(PAGE, hd),
             17 * hd + (i // 2) * (hd // 8) + 2 * (d // 16) + i % 2))


def unpack(cache):
    """Records [.., 18 hd] -> (key codes [.., 16, hd], key bytes [.., 16, hd / 16], value codes, value bytes)."""
    out = []
    for at, shift, sc in places(cache.shape[-1] // 18):
        out += [(cache[..., at] >> shift.to(torch.uint8)) & 15, cache[..., sc[:, ::GROUP]]]
    return out


def put(rec, which, i, code, byte):
    """Token i's codes [hd] and bytes [hd / 16] into a record (in place); which: 0 keys, 1 values."""
    at, shift, sc = places(rec.shape[-1] // 18)[which]
    sh = shift[i].to(torch.uint8)
    keep = ~(15 << sh.int()) & 0xff
    for o in (0, 4):                                               # (a byte twice in one index: one after the other)
        m = sh == o
        rec[at[i][m]] = ((rec[at[i][m]].int() & keep[m]) | (code[m].int() << o)).to(torch.uint8)
    rec[sc[i, ::GROUP]] = byte


def append(cache, which, x, start, cu, table, take=None):
    """Rows x (float64, already rotated) into a copy of the cache."""
    cache = cache.clone()
    byte = scale_bytes(x)
    code = codes(x, byte)
    for b in range(len(start)):
        n = int(cu[b + 1] - cu[b]) if take is None else int(take[b])
        for t in range(n):
            pos = int(start[b]) + t
            for h in range(x.shape[1]):
                r = int(cu[b]) + t
                put(cache[int(table[b, pos // PAGE]), h], which, pos % PAGE, code[r, h], byte[r, h])
    return cache


def rows(cache, table, b, start, n):
    """Keys and values [n, H, hd] of positions start.. of sequence b, float64."""
    hd = cache.shape[-1] // 18
    pages = table[b, start // PAGE:(start + n + PAGE - 1) // PAGE].long()
    kc, kb, vc, vb = unpack(cache[pages])
    out = []
    for c, s in ((kc, kb), (vc, vb)):
        x = values(c, s).transpose(1, 2).reshape(-1, cache.shape[1], hd)
        out.append(x[start % PAGE:start % PAGE + n])
    return out


def verify(q, cache, table, kn, vn, tau, lens, cu, spec, sm_scale, order, node, err):
    """Attention rows in float64 and how far a kernel's row may be off before
    its last rounding.  err: relative rounding of a query element, a new key's,
    a new value's and a weight (2^-11, or 0 for fp32); the rotation is off by
    2e-6 of a row's largest element (fp32 angles and products)."""
    Hq, Hkv, hd = q.shape[1], kn.shape[1], q.shape[2]
    G, per = Hq // Hkv, 2 if order == "paired" else 1
    out, off = torch.zeros(q.shape, dtype=F64), torch.zeros(q.shape, dtype=F64)
    for b in range(len(lens)):
        P, B = int(lens[b]), int(cu[b + 1] - cu[b])
        r = slice(per * int(cu[b]), per * int(cu[b + 1]))
        pos = P + kvq_ref.offsets(order, B, node)
        Q, KN = kvq_ref.rope(q[r], pos, spec), kvq_ref.rope(kn[r], pos, spec)
        kp, vp = rows(cache, table, b, 0, P)
        K, V = torch.cat([kp, KN]), torch.cat([vp, vn[r].to(F64)])
        fresh = torch.arange(P + per * B) >= P
        see = torch.cat([torch.ones(per * B, P, dtype=torch.bool),
                         kvq_ref.visible(order, B, tau[int(cu[b]):int(cu[b + 1])] if order == "paired" else None, node)], 1)
        for h in range(Hq):
            k, v = K[:, h // G], V[:, h // G]
            qa, ka = Q[:, h].abs(), k.abs()
            s = (Q[:, h] @ k.T * sm_scale).masked_fill(~see, -math.inf)
            p = torch.softmax(s, -1)
            size = qa @ ka.T * sm_scale
            turn = 2e-6 * sm_scale * (qa.amax(-1, keepdim=True) * ka.sum(-1) +
                                      torch.where(fresh, ka.amax(-1), 0.0) * qa.sum(-1, keepdim=True))
            d = size * (err * (1 + fresh.to(F64)) + (hd + 16) * 2.0 ** -24) + turn + 2.0 ** -20 * s.abs().clamp(max=1e4)
            d = torch.where(see, d, 0.0)
            mean = (p * d).sum(-1, keepdim=True)
            out[r, h] = p @ v
            off[r, h] = 1.2 * ((p * (d + mean + err * (1 + fresh.to(F64)) + 2.0 ** -20)) @ v.abs())
    return out, off
