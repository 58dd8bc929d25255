"""simsd_token_logprobs over the whole range of temperatures and finite logits:
parts of a row (2048 entries) that hold nothing but a mask's finite fill, and
temperatures at which c m, with c = log2(e) / T, is far beyond 2^24.  Bounds as
in test_gpu_logprobs: t carries three roundings, of the difference or of c m, of
c and its own.  (The definition takes T in 64 bits and the call in 32, 2^-25 of a
log probability.)"""
import math

import pytest
import torch

from test_gpu_logprobs import DT, check

pytestmark = pytest.mark.gpu


def masked_rows(vocab, fill, dtype):
    """Rows with whole parts, whole rows but one entry, and scattered entries at the fill."""
    g = torch.Generator().manual_seed(int(-math.log10(-fill)) + 100)
    x = torch.randn(6, vocab, generator=g) * 3
    x[0, :2048] = fill
    x[1, 2048:4096] = fill
    x[2, 4096:] = fill
    x[3] = fill
    x[3, 5000] = 1.5
    x[4] = fill
    x[5, torch.rand(vocab, generator=g) < 0.7] = fill
    return x.cuda().to(DT[dtype])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("fill", [-1e9, -1e10, -1e15, -1e20])
@pytest.mark.parametrize("temperature", [1.0, 0.3, 0.1, 0.01])
def test_parts_at_a_finite_fill(dtype, fill, temperature):
    vocab = 3 * 2048 + 77
    x = masked_rows(vocab, fill, dtype)
    check(x, [3000, 2048, 0, 5000, vocab - 1, 17], 20, temperature)
    check(x, [2047, 3000, vocab - 1, 0, 0, 4095], 3, temperature)            # (tokens at the fill, mostly)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("temperature", [1e-3, 1e-5, 1e-6, 1e-7, 1e-8, 1e-9, 1e-12, 1e-20, 1e-30, 1e12, 1e30])
def test_temperatures_of_the_whole_range(dtype, temperature):
    g = torch.Generator(device="cuda").manual_seed(9)
    x = (torch.randn(5, 5003, generator=g, device="cuda") * 4).to(DT[dtype])
    x[1] -= 12.0                                                             # a maximum near 0,
    x[2, ::7] = x[2].max()                                                   # many equal ones,
    x[3] = x[3].abs() * -1000                                                # no positive entry,
    x[4, 3000:] = -math.inf
    tokens = x.float().argmax(-1).cpu()
    check(x, tokens, 8, temperature)
    check(x, [0, 2, 7, 5002, 2999], 32, temperature)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("temperature", [4.0, 1e10, 1e30])
def test_logits_further_apart_than_the_largest_number(dtype, temperature):
    """l - M below -3.4e38, (l - M) / T inside fp32."""
    x = torch.full((3, 4500), -3e38)
    x[0, 5] = x[1, 4000] = x[1, 4400] = 3e38
    x[2] = torch.linspace(-3e38, 3e38, 4500, dtype=torch.float64).float()   # (in 32 bits its step would be infinite)
    x = x.cuda().to(DT[dtype])
    check(x, [4, 4000, 0], 20, temperature)
    check(x, [5, 17, 4499], 3, temperature)
