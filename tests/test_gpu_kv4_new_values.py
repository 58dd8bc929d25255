"""simsd_kv4_verify, bf16: new tokens whose values differ in size, up to the type's
largest beside zeros.  A token's share of the softmax does not depend on the size of
any token's values.  Bounds as in test_gpu_kv4, and each product off by 2^-32 of its
row's largest."""
import math

import pytest
import torch

import kv4_ref as ref
import speculative_decoding_diffusion_gb300 as pkg
from test_gpu_kv4 import case, close, i32, verify

pytestmark = pytest.mark.gpu


def compare(c, lens, B, order, scale):
    cache, table, cu, q, kn, vn, tau = c
    out, ws = verify(q.cuda(), cache.cuda(), table, kn.cuda(), vn.cuda(), i32(tau), lens, cu, B, dict(base=1e4), scale, order)
    assert pkg.read_status(ws) == 0
    want, off = ref.verify(q, cache, table, kn, vn, tau, lens, cu, dict(base=1e4), scale, order, 0, 2.0 ** -11)
    per, extra = 2 if order == "paired" else 1, torch.zeros_like(off)
    for b, P in enumerate(lens):                                              # of the largest value that the row may see
        r = slice(per * int(cu[b]), per * int(cu[b + 1]))
        extra[r] = (P + 64) * 2.0 ** -32 * max(12.0, float(vn[r].abs().max()))
    close(out, want, off + extra, "bf16")


@pytest.mark.parametrize("big", [1e10, 1e24, 3e38])
@pytest.mark.parametrize("B", [2, 4, 8, 16, 32])
@pytest.mark.parametrize("lens", [(0, 0), (33, 700)])
def test_zero_values_beside_large_ones(B, big, lens):
    """Half of the new tokens hold zeros, or values of their own size; the others hold values of about `big`."""
    c = case(B, lens, [B] * 2, "causal", "bf16", 4, 2, 128)
    vn = c[5]
    vn[0::2] = 0.0
    vn[1::2] = (vn[1::2].float().clamp(-1.1, 1.1) * (big / 1.15)).bfloat16()
    compare(c, lens, B, "causal", 0.1)


@pytest.mark.parametrize("order,B", [("causal", 2), ("paired", 2), ("paired", 8), ("paired", 16)])
def test_values_of_every_size(order, B):
    """Each new token's values of another size, 2^-60 to 2^127."""
    lens = (0, 40)
    c = case(B, lens, [B] * 2, order, "bf16", 4, 1, 64)
    vn = c[5]
    size = torch.linspace(-60, 126, vn.shape[0])[torch.randperm(vn.shape[0], generator=torch.Generator().manual_seed(B))].round()
    vn.copy_((vn.double().clamp(-1.9, 1.9) * torch.exp2(size.double())[:, None, None]).bfloat16())
    compare(c, lens, B, order, 0.1)


@pytest.mark.parametrize("big", [1.0, 1e30, 3e38])
@pytest.mark.parametrize("B,lens", [(1, (4096, 900)), (2, (4096, 16)), (4, (4096, 900)), (8, (3000, 900)), (16, (20000, 900)), (32, (4096, 77))])
def test_prompts_beside_large_values(B, lens, big):
    """A new token 17 log2 units above every key of the prompt: thousands of those make up a few hundredths of the sum,
    whatever its values are."""
    cache, table, cu, q, kn, vn, tau = case(B, lens, [B] * 2, "causal", "bf16", 4, 1, 128)
    cache[..., 16 * 128:17 * 128] = cache[..., 16 * 128:17 * 128].clamp(max=0x30)        # keys of 2^-9 and less, scores near 0
    u = torch.randn(128, generator=torch.Generator().manual_seed(1)).sign().bfloat16()
    q.copy_(u.expand_as(q))
    kn.copy_((u * 0.92).bfloat16().expand_as(kn))                                        # the row's own: 128 * 0.92 * 0.1 nats
    vn.copy_((vn.float().clamp(-1.1, 1.1) * (big / 1.15)).bfloat16())
    vn[1::2] = 0.0
    compare((cache, table, cu, q, kn, vn, tau), lens, B, "causal", 0.1)
