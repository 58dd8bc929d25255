"""simsd_token_logprobs at sizes past one step of its loops: more parts and segments
than a CTA has threads, more rows than two a SM, rows further apart than 32 bits
count.  Bounds as in test_gpu_logprobs."""
import math

import pytest
import torch

import speculative_decoding_diffusion_gb300 as pkg
from test_gpu_logprobs import DT, call, check, definition, near

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("vocab,rows", [(2 ** 21, 2), (2 ** 21 - 3, 1), (600001, 3), (262145, 4)])
def test_long_rows(dtype, vocab, rows):
    g = torch.Generator(device="cuda").manual_seed(vocab)
    x = (torch.randn(rows, vocab, generator=g, device="cuda") * 3).to(DT[dtype])
    x[0, 100000:230000] = -math.inf
    tokens = torch.randint(0, vocab, (rows,), generator=torch.Generator().manual_seed(rows))
    check(x, tokens, 32)
    check(x, x.float().argmax(-1).cpu(), 1, 0.25)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("vocab,top", [(1, 1), (31, 31), (300, 32), (5000, 20), (33000, 32), (151936, 20)])
def test_many_rows(dtype, vocab, top):
    rows = 347
    g = torch.Generator(device="cuda").manual_seed(vocab + top)
    x = (torch.randn(rows, vocab, generator=g, device="cuda") * 3).to(DT[dtype])
    x[5], x[6, : vocab // 2] = 2.0, -math.inf
    tokens = torch.randint(0, vocab, (rows,), generator=torch.Generator().manual_seed(top))
    tokens[6] = vocab - 1
    check(x, tokens, top)


def test_rows_past_32_bit_offsets():
    vocab, stride = 3001, 2 ** 31 + 9
    flat = torch.empty(2 * stride + vocab, dtype=torch.bfloat16, device="cuda")
    x = flat.as_strided((3, vocab), (stride, 1))
    x.copy_(torch.randn(3, vocab, generator=torch.Generator().manual_seed(1)) * 3)
    got, ws = call(x, [0, 3000, 17], 5)
    want = definition(x.clone(), [0, 3000, 17], 5)
    assert pkg.read_status(ws) == 0 and torch.equal(got["rank"].long(), want["rank"])
    assert torch.equal(got["top_ids"].long(), want["top_ids"])
    for k in ("logprob", "entropy", "top_logprobs"):
        near(got[k], want[k])
