"""Plain 64-bit forms of the 8-bit-cache operators, sequence by sequence, for
their tests: rotary positions, the page map, the append and the attention.
All on the CPU; a page and head's scale is held as its exponent byte."""
import math

import torch

PAGE = 16
F64 = torch.float64


def freqs(hd, base=1.0e4, rotary_dim=0, scaling="plain", factor=1.0, original_len=0, fast=32.0,
          slow=1.0, attn_factor=0.0, interleaved=False):
    rd = rotary_dim or hd
    out = []
    for i in range(rd // 2):
        w = base ** (-2.0 * i / rd)
        if scaling == "linear":
            w /= factor
        elif scaling == "ntk":
            w = (base * factor ** (rd / (rd - 2.0))) ** (-2.0 * i / rd)
        elif scaling == "yarn":
            lo = max(0, math.floor(rd * math.log(original_len / (2 * math.pi * fast)) / (2 * math.log(base))))
            hi = min(rd - 1, math.ceil(rd * math.log(original_len / (2 * math.pi * slow)) / (2 * math.log(base))))
            r = min(1.0, max(0.0, (i - lo) / max(hi - lo, 0.001)))
            w = w * (1 - r) + w / factor * r
        elif scaling == "banded":
            r = min(1.0, max(0.0, (original_len * w / (2 * math.pi) - slow) / (fast - slow)))
            w = w / factor * (1 - r) + w * r
        out.append(w)
    mul = attn_factor or (0.1 * math.log(factor) + 1 if scaling == "yarn" else 1.0)
    return torch.tensor(out, dtype=F64), mul


def rope(x, pos, spec, inverse=False):
    """x [rows, heads, hd] (any type) -> float64, rotated."""
    x = x.to(F64)
    w, mul = freqs(x.shape[-1], **spec)
    a = pos.to(F64)[:, None] * w
    c, s = (a.cos() * mul)[:, None], (a.sin() * mul * (-1 if inverse else 1))[:, None]
    h = len(w)
    y = x.clone()
    one, two = (slice(0, 2 * h, 2), slice(1, 2 * h, 2)) if spec.get("interleaved") else (slice(0, h), slice(h, 2 * h))
    y[..., one] = x[..., one] * c - x[..., two] * s
    y[..., two] = x[..., two] * c + x[..., one] * s
    return y


def code(y):
    """Nearest e4m3 value, ties to even, saturating (float64 in and out)."""
    y = y.clamp(-448.0, 448.0)
    _, e = torch.frexp(y)
    step = torch.exp2((e - 4).clamp(min=-9).to(F64))
    return torch.round(y / step) * step


def exponent(amax):
    """Smallest E in -64..7 with amax <= 448 * 2^E."""
    for e in range(-64, 8):
        if amax <= 448.0 * 2.0 ** e:
            return e
    return 7


def e4m3_values(codes):
    """uint8 codes -> float64 values."""
    return codes.view(torch.float8_e4m3fn).to(torch.float32).to(F64)


def append(x, start, cu, table, codes, scale, take=None):
    """Rows x (float64, already rotated) into copies of the page arrays:
    values [pages, H, 16, hd] (codes as the values they are) and exponent
    bytes.  Returns (code values, exponent bytes)."""
    val, byte = e4m3_values(codes), scale.clone()
    for b in range(len(start)):
        n = int(cu[b + 1] - cu[b]) if take is None else int(take[b])
        s0 = int(start[b])
        for pg in range(s0 // PAGE, (s0 + n + PAGE - 1) // PAGE if n else 0):
            page = int(table[b, pg])
            lo, hi = max(0, s0 - pg * PAGE), min(PAGE, s0 + n - pg * PAGE)
            rows = x[int(cu[b]) + pg * PAGE + lo - s0:int(cu[b]) + pg * PAGE + hi - s0]
            for h in range(x.shape[1]):
                new = rows[:, h]
                e, was = exponent(float(new.abs().max())), int(byte[page, h])
                odd = not bool(torch.isfinite(new).all()) or (lo > 0 and was == 255)
                if lo > 0 and not odd:
                    e = max(e, min(max(was - 127, -64), 7))
                    val[page, h, :lo] = code(val[page, h, :lo] * 2.0 ** (was - 127 - e))
                val[page, h, lo:hi] = code(new * 2.0 ** -e)
                byte[page, h] = 255 if odd else e + 127
    return val, byte


def visible(order, B, tau, node):
    """[n, n] truth values: row r sees new token c."""
    n = 2 * B if order == "paired" else B
    m = torch.zeros(n, n, dtype=torch.bool)
    for r in range(n):
        for c in range(n):
            if order == "causal":
                m[r, c] = c <= r
            elif order == "nodes":
                m[r, c] = r // node == c // node
            elif r >= B:
                m[r, c] = tau[c - B] >= tau[r - B] if c >= B else tau[c] < tau[r - B]
            else:
                m[r, c] = c < B and bool(tau[c] <= tau[r])
    return m


def offsets(order, B, node):
    n = 2 * B if order == "paired" else B
    i = torch.arange(n)
    return i % B if order == "paired" else i % node if order == "nodes" else i


def verify(q, k_codes, v_codes, k_scale, v_scale, table, kn, vn, tau, lens, cu, spec, sm_scale, order,
           node, q_err, p_err):
    """Attention rows in float64 and how far a kernel's row may be off before
    its last rounding: query elements off by q_err of themselves, weights by
    p_err, sums over hd in fp32."""
    Hq, Hkv, hd = q.shape[1], kn.shape[1], q.shape[2]
    G, per = Hq // Hkv, 2 if order == "paired" else 1
    out = torch.zeros(q.shape, dtype=F64)
    off = torch.zeros(q.shape, dtype=F64)
    for b in range(len(lens)):
        P, B = int(lens[b]), int(cu[b + 1] - cu[b])
        r = slice(per * int(cu[b]), per * int(cu[b + 1]))
        pos = P + offsets(order, B, node)
        Q, KN = rope(q[r], pos, spec), rope(kn[r], pos, spec)
        page = table[b, :(P + PAGE - 1) // PAGE].long()

        def past(codes, scale):
            x = e4m3_values(codes[page]) * torch.exp2(scale[page].to(F64) - 127)[..., None, None]
            x[scale[page] == 255] = math.nan
            return x.permute(0, 2, 1, 3).reshape(-1, Hkv, hd)[:P]

        K = torch.cat([past(k_codes, k_scale), KN])
        V = torch.cat([past(v_codes, v_scale), vn[r].to(F64)])
        see = torch.cat([torch.ones(per * B, P, dtype=torch.bool),
                         visible(order, B, tau[int(cu[b]):int(cu[b + 1])] if order == "paired" else None, node)], 1)
        for h in range(Hq):
            k, v = K[:, h // G], V[:, h // G]
            s = (Q[:, h] @ k.T * sm_scale).masked_fill(~see, -math.inf)
            p = torch.softmax(s, -1)
            size = Q[:, h].abs() @ k.abs().T * sm_scale
            d = size * (q_err + (hd + 16) * 2.0 ** -24) + 2.0 ** -20 * s.abs().clamp(max=1e4)
            d = torch.where(see, d, 0.0)
            mean = (p * d).sum(-1, keepdim=True)
            out[r, h] = p @ v
            off[r, h] = 1.2 * ((p * (d + mean + p_err + 2.0 ** -20)) @ v.abs())
    return out, off
