"""Host side of the 8-bit-cache calls beyond test_kvq_host: calls without
rows (no GPU needed, no kernel launched)."""
import ctypes

import pytest

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
