"""simsd_rope against the rotation in 64 bits.

Tolerance of an element y = mul (x1 cos - x2 sin): the angle is off by at
most ~6e-7 rad and cos, sin, mul and the two products round by 2^-24 each,
so 1.5e-6 mul (|x1| + |x2|) covers it; bf16 output adds half a step, 2^-8 |y|
(torch.finfo.eps / 2)."""
import pytest
import torch

import kvq_ref as ref
import speculative_decoding_diffusion_gb300 as pkg
from speculative_decoding_diffusion_gb300 import binding

pytestmark = pytest.mark.gpu

SCALED = {"plain": {}, "linear": dict(factor=4.0), "ntk": dict(factor=4.0),
          "yarn": dict(factor=8.0, original_len=4096), "banded": dict(factor=8.0, original_len=8192, fast=4.0)}


def close(got, x, pos, spec, inverse=False):
    want = ref.rope(x, pos, spec, inverse)
    _, mul = ref.freqs(x.shape[-1], **spec)
    h = (spec.get("rotary_dim") or x.shape[-1]) // 2
    a = x.double().abs()
    size = torch.zeros_like(a)
    one, two = (slice(0, 2 * h, 2), slice(1, 2 * h, 2)) if spec.get("interleaved") else (slice(0, h), slice(h, 2 * h))
    size[..., one] = size[..., two] = a[..., one] + a[..., two]
    off = 1.5e-6 * mul * size + (2.0 ** -8 * want.abs() if got.dtype == torch.bfloat16 else 0.0)
    assert ((got.cpu().double() - want).abs() <= off).all()


@pytest.mark.parametrize("scaling", list(SCALED))
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dtype,hd,rd", [(torch.bfloat16, 128, 0), (torch.bfloat16, 64, 16), (torch.float32, 64, 0),
                                         (torch.float32, 128, 50), (torch.bfloat16, 128, 24), (torch.bfloat16, 64, 2)])
def test_matches_definition(dtype, hd, rd, interleaved, scaling):
    if scaling == "ntk" and rd == 2:
        rd = 4
    spec = dict(base=1.0e6, rotary_dim=rd, interleaved=interleaved, scaling=scaling, **SCALED[scaling])
    g = torch.Generator().manual_seed(hd + rd)
    for rows, hq, hkv in ((1, 1, 1), (37, 12, 3)):
        x, k = torch.randn(rows, hq, hd, generator=g).to(dtype), torch.randn(rows, hkv, hd, generator=g).to(dtype)
        pos = torch.randint(0, 40000, (rows,), generator=g, dtype=torch.int32)
        for inverse in (False, True):
            y, ky = torch.empty_like(x, device="cuda"), torch.empty_like(k, device="cuda")
            pkg.rope(x.cuda(), pos.cuda(), pkg.rope_spec(**spec), y, k.cuda(), ky, inverse=inverse)
            close(y, x, pos, spec, inverse)
            close(ky, k, pos, spec, inverse)


@pytest.mark.parametrize("rows", [1, 5, 303, 457, 607, 2433])
def test_row_counts_around_the_rows_of_a_cta(rows):
    spec = dict(base=1.0e4)
    x = torch.randn(rows, 2, 64, generator=torch.Generator().manual_seed(rows))
    pos = torch.arange(rows, dtype=torch.int32)
    y = torch.empty_like(x, device="cuda")
    pkg.rope(x.cuda(), pos.cuda(), pkg.rope_spec(**spec), y)
    close(y, x, pos, spec)


def test_far_and_negative_positions():
    spec = dict(base=1.0e4)
    pos = torch.tensor([0, -1, 1, 2 ** 24 - 1, 2 ** 24, 2 ** 24 + 1, -(2 ** 24), 2 ** 30, -(2 ** 30)], dtype=torch.int32)
    x = torch.randn(len(pos), 3, 128, generator=torch.Generator().manual_seed(1))
    y = torch.empty_like(x, device="cuda")
    pkg.rope(x.cuda(), pos.cuda(), pkg.rope_spec(**spec), y)
    close(y, x, pos, spec)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("shift", [0, 1])
def test_strides_in_place_and_unaligned(dtype, shift):
    """Queries and keys inside fused rows, rotated in place; with shift 1 the
    rows start off a 16-byte boundary (element-wise path).  What lies between
    the heads stays as it was."""
    T, hq, hkv, hd = 33, 6, 2, 128
    spec = dict(base=1.0e4, interleaved=bool(shift))
    g = torch.Generator().manual_seed(3)
    buf = torch.randn(T * (hq + 2 * hkv) * hd + shift, generator=g).to(dtype)
    dev = buf.cuda()
    rows, host = (t[shift:].view(T, hq + 2 * hkv, hd) for t in (dev, buf))
    pos = torch.randint(0, 9000, (T,), generator=g, dtype=torch.int32)
    q, k = rows[:, :hq], rows[:, hq:hq + hkv]
    pkg.rope(q, pos.cuda(), pkg.rope_spec(**spec), q, k, k)
    close(q, host[:, :hq], pos, spec)
    close(k, host[:, hq:hq + hkv], pos, spec)
    assert torch.equal(rows[:, hq + hkv:].cpu(), host[:, hq + hkv:])


def test_heads_first_layout_and_gradient():
    """[heads, rows, hd] storage, and the inverse as the gradient: <g, R x> =
    <R' g, x>, and against central differences of the 64-bit form."""
    H, T, hd = 5, 21, 64
    spec = dict(base=1.0e4, rotary_dim=32, scaling="yarn", factor=4.0, original_len=64)
    g = torch.Generator().manual_seed(4)
    x = torch.randn(H, T, hd, generator=g)
    up = torch.randn(T, H, hd, generator=g)
    pos = torch.arange(T, dtype=torch.int32)
    y = torch.empty(T, H, hd, device="cuda")
    pkg.rope(x.cuda().transpose(0, 1), pos.cuda(), pkg.rope_spec(**spec), y)
    close(y, x.transpose(0, 1), pos, spec)
    dx = torch.empty(H, T, hd, device="cuda")
    pkg.rope(up.cuda(), pos.cuda(), pkg.rope_spec(**spec), dx.transpose(0, 1), inverse=True)
    xt = x.transpose(0, 1).double().contiguous()
    for r, h, d in ((0, 0, 0), (7, 2, 5), (20, 4, 31), (13, 1, 40)):
        e = torch.zeros_like(xt)
        e[r, h, d] = 1e-4
        slope = ((ref.rope(xt + e, pos, spec) - ref.rope(xt - e, pos, spec)) / 2e-4 * up.double()).sum()
        assert abs(float(dx[h, r, d]) - float(slope)) <= 1e-5
    lhs = (up.double() * y.cpu().double()).sum()
    rhs = (dx.cpu().double().transpose(0, 1) * xt).sum()
    assert abs(lhs - rhs) <= 1e-6 * (up.double().abs() * y.cpu().double().abs()).sum()


def test_graph_replay_and_other_stream():
    spec = pkg.rope_spec(base=1.0e4)
    x = torch.randn(64, 4, 128, device="cuda")
    pos = torch.arange(64, dtype=torch.int32, device="cuda")
    y, z = torch.empty_like(x), torch.empty_like(x)
    pkg.rope(x, pos, spec, z)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        pkg.rope(x, pos, spec, y)
    for seed in (1, 2):
        x.normal_(generator=torch.Generator("cuda").manual_seed(seed))
        graph.replay()
        pkg.rope(x, pos, spec, z)
        assert torch.equal(y, z)


def test_refusals():
    x = torch.zeros(4, 2, 64, device="cuda")
    pos = torch.zeros(4, dtype=torch.int32, device="cuda")
    ok = pkg.rope_spec(base=1.0e4)
    with pytest.raises(ValueError):
        pkg.rope(x, pos.cpu(), ok, x)
    with pytest.raises(ValueError):
        pkg.rope(x, pos[:3], ok, x)
    with pytest.raises(TypeError):
        pkg.rope(x, pos.long(), ok, x)
    with pytest.raises(TypeError):
        pkg.rope(x.half(), pos, ok, x.half())
    with pytest.raises(pkg.SimsdError):
        pkg.rope(x, pos, pkg.rope_spec(base=0.5), x)
    assert binding.SIMSD_ROPE_HALF == 0
