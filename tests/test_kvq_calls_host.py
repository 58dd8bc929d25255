"""Host side of the 8-bit-cache calls beyond test_kvq_host: calls without
rows, types of the cache, layouts of an output (no GPU needed, no kernel launched)."""
import ctypes

import pytest
import torch

from speculative_decoding_diffusion_gb300 import binding
from test_kvq_host import append_desc, rope_desc


@pytest.fixture(scope="module")
def lib():
    from speculative_decoding_diffusion_gb300 import build
    build.build()
    return binding.lib()


def test_calls_without_rows_need_no_arrays(lib):
    """A tensor without elements has no memory: its pointer is NULL."""
    none = dict(x0=None, y0=None, x1=None, y1=None, positions=None)
    assert lib.simsd_rope(ctypes.byref(rope_desc(rows=0, **none)), None) == 0
    assert lib.simsd_rope(ctypes.byref(rope_desc(rows=0, head_dim=96, **none)), None) == 2
    assert lib.simsd_kvq_append(ctypes.byref(append_desc(total_n=0, k=None, v=None)), None) == 0
    assert lib.simsd_kvq_append(ctypes.byref(append_desc(total_n=0, k=None, v=None, start=None)), None) == 1


@pytest.mark.parametrize("which", ["k_cache", "v_cache", "k_scale", "v_scale"])
def test_a_cache_of_another_8_bit_type_is_refused(which):
    """e5m2 codes, codes in the scales' type and scales in the codes', truth values."""
    bytes_ = dict(k_cache=torch.zeros(3, 2, 16, 64, dtype=torch.uint8), v_cache=torch.zeros(3, 2, 16, 64, dtype=torch.uint8),
                  k_scale=torch.zeros(3, 2, dtype=torch.uint8), v_scale=torch.zeros(3, 2, dtype=torch.uint8))
    mine, other = torch.float8_e4m3fn, torch.float8_e8m0fnu
    if which.endswith("scale"):
        mine, other = other, mine
    for dtype in (torch.float8_e5m2, torch.float8_e4m3fnuz, other, torch.bool, torch.float32):
        with pytest.raises(TypeError):
            binding._codes(**dict(bytes_, **{which: bytes_[which].to(torch.float32) if dtype == torch.float32
                                             else bytes_[which].view(dtype)}))
    for dtype in (mine, torch.uint8, torch.int8):
        binding._codes(**dict(bytes_, **{which: bytes_[which].view(dtype)}))

    # through a call: the type is seen before the device
    q, ids, spec = torch.zeros(4, 2, 64), torch.zeros(5, dtype=torch.int32), binding.rope_spec()
    bad = dict(bytes_, **{which: bytes_[which].view(torch.float8_e5m2)})
    with pytest.raises(TypeError):
        binding.kvq_append(q, q, ids[:1], ids[:2], *bad.values(), ids[:1].view(1, 1), ids, spec)
    with pytest.raises(TypeError):
        binding.kvq_verify(q, *bad.values(), ids[:1].view(1, 1), q, q, None, ids[:1], ids[:2], q, ids, 4, 4, spec, 1.0,
                           order=binding.SIMSD_ORDER_CAUSAL)


def test_heads_that_share_memory_are_found():
    """Against every pair of heads compared, strides of every relation to hd, rows and heads."""
    hd = 4
    for rows in (0, 1, 2, 3, 5):
        for heads in (1, 2, 3, 4):
            for row in range(0, 26):
                for head in range(0, 26):
                    at = [r * row + h * head for r in range(rows) for h in range(heads)]
                    want = all(abs(a - b) >= hd for i, a in enumerate(at) for b in at[:i])
                    got = binding._apart(rows, heads, hd, row, head)
                    assert got == want, (rows, heads, row, head)
    assert binding._apart(7, 3, 64, 3 * 64, 64) and binding._apart(7, 3, 64, 64, 7 * 64)
    assert not binding._apart(7, 3, 64, 0, 64) and not binding._apart(7, 3, 64, 64, 0)
