"""simsd_kvq_append, code by code, rotated keys included.

The kernel's rotated element is off the exact x1 cos - x2 sin by less than
e = 2e-6 mul (|x1| + |x2|): the page's first angle 3e-7, the turn from there (up
to four tabled angles of 1.2e-7 and three products of 1.7e-7) 1e-6, their
product, the factor and the rotation's own three roundings 4e-7 together.  So
  the scale is one that a maximum within the elements' e would get, and
  a code is one that a value within e of the exact one would get
(elements that are not rotated, and values: e = 0), older codes are the old
values' nearest at the scale found, and everything else is as it was."""
import pytest
import torch

import kvq_ref as ref
import speculative_decoding_diffusion_gb300 as pkg
from test_gpu_kvq import DT, PAGE, Cache, cu_of, put, tables

pytestmark = pytest.mark.gpu
F64 = torch.float64


def check_codes(x, e, start, n, take, table, before, scale_before, after, scale_after):
    """x exact [rows, H, hd], e how far the kernel's may be off."""
    H, cu = x.shape[1], cu_of(n)
    old, got = ref.e4m3_values(before), ref.e4m3_values(after)
    untouched = torch.ones(before.shape, dtype=torch.bool)
    pages_kept = torch.ones(scale_before.shape, dtype=torch.bool)
    for b in range(len(start)):
        s0, m = start[b], n[b] if take is None else take[b]
        for pg in range(s0 // PAGE, (s0 + m + PAGE - 1) // PAGE if m else 0):
            page, first = int(table[b, pg]), pg * PAGE
            lo, hi = max(0, s0 - first), min(PAGE, s0 + m - first)
            r = slice(int(cu[b]) + first + lo - s0, int(cu[b]) + first + hi - s0)
            for h in range(H):
                y, d, was, byte = x[r, h], e[r, h], int(scale_before[page, h]), int(scale_after[page, h])
                ends = [ref.exponent(float((y.abs() - d).max().clamp(min=0))), ref.exponent(float((y.abs() + d).max()))]
                if lo > 0:
                    ends = [max(z, min(max(was - 127, -64), 7)) for z in ends]
                E = byte - 127
                assert ends[0] <= E <= ends[1], (b, pg, h, E, ends)
                new = got[page, h, lo:hi]
                assert (new >= ref.code((y - d) * 2.0 ** -E)).all() and (new <= ref.code((y + d) * 2.0 ** -E)).all(), (b, pg, h)
                assert torch.equal(got[page, h, :lo], ref.code(old[page, h, :lo] * 2.0 ** (was - 127 - E))), (b, pg, h)
                untouched[page, h, :hi] = pages_kept[page, h] = False
    assert torch.equal(before[untouched], after[untouched]) and torch.equal(scale_before[pages_kept], scale_after[pages_kept])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("hd,H,spec", [(128, 2, dict(base=1e4)), (64, 3, dict(base=1e4, interleaved=True, rotary_dim=32)),
                                       (128, 1, dict(base=1e6, rotary_dim=50)), (64, 2, dict(base=1e6, rotary_dim=24, interleaved=True)),
                                       (128, 1, dict(base=1e6, scaling="yarn", factor=4.0, original_len=64))])
@pytest.mark.parametrize("far", [0, 40000])
def test_codes(dtype, hd, H, spec, far):
    """Sizes that differ from row to row, pages half full of older codes of other scales, far positions, the first rows taken."""
    g = torch.Generator().manual_seed(hd + H + far)
    n = [int(i) for i in torch.randint(0, 90, (40,), generator=g)]
    start = [int(i) for i in torch.randint(0, 60, (40,), generator=g)]
    take = [int(m * f) for m, f in zip(n, torch.rand(40, generator=g).tolist())] if far else None
    table, total = tables(g, [(s + m + PAGE - 1) // PAGE for s, m in zip(start, n)])
    if far:                                              # the same pages, behind entries that are not read
        start = [s + far for s in start]
        table = torch.cat([torch.full((40, far // PAGE), 2 ** 30), table], 1)
    c = Cache(g, total, H, hd, 110, 126)
    rows = sum(n)
    size = torch.exp2(torch.randint(-4, 5, (rows, H, 1), generator=g).float())
    k, v = ((torch.randn(rows, H, hd, generator=g) * size).to(DT[dtype]) for _ in range(2))
    dev = c.cuda()
    assert pkg.read_status(put(k.cuda(), v.cuda(), start, n, table, dev, spec, take)) == 0
    got = [t.cpu() for t in dev]
    pos = torch.cat([torch.arange(s, s + m) for s, m in zip(start, n)])
    x, (w, mul) = ref.rope(k, pos, spec), ref.freqs(hd, **spec)
    a, e, half = k.to(F64).abs(), torch.zeros(rows, H, hd, dtype=F64), len(w)
    one, two = (slice(0, 2 * half, 2), slice(1, 2 * half, 2)) if spec.get("interleaved") else (slice(0, half), slice(half, 2 * half))
    e[..., one] = e[..., two] = 2e-6 * mul * (a[..., one] + a[..., two])
    check_codes(x, e, start, n, take, table, c.k, c.ks, got[0], got[2])
    check_codes(v.to(F64), torch.zeros_like(e), start, n, take, table, c.v, c.vs, got[1], got[3])
