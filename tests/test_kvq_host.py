"""Host-side checks of the 8-bit-cache calls (no GPU needed, no kernel
launched): descriptor layouts, refusals before any launch, workspace sizes."""
import ctypes
import os
import subprocess

import pytest
import torch

from speculative_decoding_diffusion_gb300 import binding

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE = 1 << 40          # never dereferenced: the calls return before launching
DESCS = {"simsd_rope_spec": binding.RopeSpec, "simsd_rope_desc": binding.RopeDesc,
         "simsd_page_map_desc": binding.PageMapDesc, "simsd_kvq_append_desc": binding.KvqAppendDesc,
         "simsd_kvq_verify_desc": binding.KvqVerifyDesc}


@pytest.fixture(scope="module")
def lib():
    from speculative_decoding_diffusion_gb300 import build
    build.build()
    return binding.lib()


def test_descriptor_layouts_match_the_header(tmp_path):
    lines = ['#include <stddef.h>', '#include <stdio.h>', '#include "simsd.h"', 'int main(void) {']
    for cname, py in DESCS.items():
        lines.append('  printf("%s . %%zu\\n", sizeof(%s));' % (cname, cname))
        for f, _ in py._fields_:
            lines.append('  printf("%s %s %%zu\\n", offsetof(%s, %s));' % (cname, f, cname, f))
    src, exe = tmp_path / "l.c", tmp_path / "l"
    src.write_text("\n".join(lines + ["  return 0;", "}"]))
    subprocess.run(["gcc", "-std=c11", "-Wall", "-Werror", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)],
                   check=True)
    for line in subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.splitlines():
        cname, f, at = line.split()
        py = DESCS[cname]
        assert int(at) == (ctypes.sizeof(py) if f == "." else getattr(py, f).offset), (cname, f)


def fill(d, **kw):
    for k, v in kw.items():
        setattr(d, k, v)
    return d


GOOD_SPEC = dict(base=1e4)


def rope_desc(**kw):
    d = fill(binding.RopeDesc(), rows=4, num_heads0=2, num_heads1=1, head_dim=64, dtype=1,
             rope=binding.rope_spec(**GOOD_SPEC), positions=FAKE, x0=FAKE, y0=FAKE, x1=FAKE, y1=FAKE)
    return fill(d, **kw)


@pytest.mark.parametrize("bad,code", [
    (dict(rows=-1), 2), (dict(num_heads0=0), 2), (dict(num_heads0=16385), 2), (dict(num_heads1=-1), 2), (dict(head_dim=96), 2),
    (dict(inverse=2), 2), (dict(dtype=2), 4), (dict(positions=None), 1), (dict(x0=None), 1), (dict(y1=None), 1),
    (dict(x0=FAKE + 1), 8), (dict(y0=FAKE + 1), 8)])
def test_rope_refusals(lib, bad, code):
    assert lib.simsd_rope(ctypes.byref(rope_desc(**bad)), None) == code
    assert lib.simsd_rope(None, None) == 1


def test_rope_without_rows_is_nothing(lib):
    assert lib.simsd_rope(ctypes.byref(rope_desc(rows=0)), None) == 0


NAN, INF = float("nan"), float("inf")


@pytest.mark.parametrize("bad", [
    dict(base=1.0), dict(base=NAN), dict(base=INF), dict(rotary_dim=3), dict(rotary_dim=66), dict(rotary_dim=-2), dict(style=2),
    dict(scaling=5), dict(scaling=-1), dict(scaling=1, factor=0.5), dict(scaling=1, factor=NAN), dict(scaling=2, factor=INF),
    dict(scaling=2, factor=2.0, rotary_dim=2), dict(scaling=3, factor=2.0, original_len=0),
    dict(scaling=3, factor=2.0, original_len=64, fast=1.0, slow=1.0), dict(scaling=4, factor=2.0, original_len=64, slow=0.0),
    dict(scaling=4, factor=2.0, original_len=64, fast=INF), dict(attn_factor=-1.0), dict(attn_factor=NAN)])
def test_rotary_numbers_out_of_range(lib, bad):
    spec = fill(binding.rope_spec(**GOOD_SPEC), **bad)
    assert lib.simsd_rope(ctypes.byref(rope_desc(rope=spec)), None) == 2
    assert lib.simsd_kvq_append(ctypes.byref(append_desc(rope=spec)), None) == 2
    assert lib.simsd_kvq_verify(ctypes.byref(verify_desc(rope=spec)), None) == 2
    assert lib.simsd_kvq_verify_workspace_size(ctypes.byref(verify_desc(rope=spec))) == 0


def test_unknown_scaling_name():
    with pytest.raises(ValueError):
        binding.rope_spec(scaling="stretched")


def map_desc(**kw):
    d = fill(binding.PageMapDesc(), batch=4, page_size=16, num_pages=100, max_pages_per_seq=8, total_n=10, workspace=FAKE,
             workspace_bytes=256, **{f: FAKE for f in ("lens", "cu_n", "held", "queue", "free_pages", "block_table", "held_out",
                                                       "queue_out", "served", "slots")})
    return fill(d, **kw)


@pytest.mark.parametrize("bad,code", [
    (dict(batch=0), 2), (dict(batch=16385), 2), (dict(page_size=32), 2), (dict(num_pages=0), 2), (dict(num_pages=1 << 30), 2),
    (dict(max_pages_per_seq=0), 2), (dict(max_pages_per_seq=1 << 29), 2), (dict(total_n=-1), 2), (dict(lens=None), 1),
    (dict(cu_n=None), 1), (dict(held=None), 1), (dict(queue=None), 1), (dict(free_pages=None), 1), (dict(block_table=None), 1),
    (dict(held_out=None), 1), (dict(queue_out=None), 1), (dict(served=None), 1), (dict(workspace=None), 5),
    (dict(workspace=FAKE + 8), 5), (dict(workspace_bytes=255), 5)])
def test_page_map_refusals(lib, bad, code):
    d = map_desc(**bad)
    assert lib.simsd_page_map(ctypes.byref(d), None) == code
    assert (lib.simsd_page_map_workspace_size(ctypes.byref(d)) == 0) == (code == 2)
    assert lib.simsd_page_map(None, None) == 1 and lib.simsd_page_map_workspace_size(None) == 0


def append_desc(**kw):
    d = fill(binding.KvqAppendDesc(), batch=2, num_kv_heads=2, head_dim=64, page_size=16, num_pages=9, max_pages_per_seq=4,
             total_n=8, dtype=1, rope=binding.rope_spec(**GOOD_SPEC), workspace=FAKE, workspace_bytes=256,
             **{f: FAKE for f in ("k", "v", "start", "cu_n", "k_cache", "v_cache", "k_scale", "v_scale", "block_table")})
    return fill(d, **kw)


@pytest.mark.parametrize("bad,code", [
    (dict(batch=0), 2), (dict(num_kv_heads=0), 2), (dict(num_kv_heads=1025), 2), (dict(head_dim=80), 2), (dict(page_size=8), 2),
    (dict(num_pages=0), 2), (dict(max_pages_per_seq=0), 2), (dict(total_n=-1), 2), (dict(k_row=-128), 2), (dict(dtype=3), 4),
    (dict(k=None), 1), (dict(v=None), 1), (dict(start=None), 1), (dict(cu_n=None), 1), (dict(k_cache=None), 1),
    (dict(v_scale=None), 1), (dict(block_table=None), 1), (dict(k=FAKE + 2), 8), (dict(v_cache=FAKE + 8), 8), (dict(k_row=132), 8),
    (dict(v_row=130), 8), (dict(workspace=None), 5), (dict(workspace=FAKE + 128), 5), (dict(workspace_bytes=4), 5)])
def test_append_refusals(lib, bad, code):
    assert lib.simsd_kvq_append(ctypes.byref(append_desc(**bad)), None) == code
    assert lib.simsd_kvq_append(None, None) == 1


def test_append_of_nothing(lib):
    assert lib.simsd_kvq_append(ctypes.byref(append_desc(total_n=0)), None) == 0


def verify_desc(**kw):
    d = fill(binding.KvqVerifyDesc(), batch=2, num_q_heads=4, num_kv_heads=2, head_dim=64, page_size=16, num_pages=9,
             max_pages_per_seq=4, total_B=8, B_max=4, dtype=1, rope=binding.rope_spec(**GOOD_SPEC), sm_scale=1.0, workspace=FAKE,
             workspace_bytes=1 << 40,
             **{f: FAKE for f in ("q", "k_cache", "v_cache", "k_scale", "v_scale", "block_table", "k_new", "v_new", "tau", "lens",
                                  "cu_B", "out")})
    return fill(d, **kw)


@pytest.mark.parametrize("bad,code", [
    (dict(batch=0), 2), (dict(num_q_heads=3), 2), (dict(num_kv_heads=0), 2), (dict(head_dim=32), 2), (dict(page_size=64), 2),
    (dict(num_pages=0), 2), (dict(max_pages_per_seq=0), 2), (dict(B_max=0), 2), (dict(B_max=33, total_B=40), 2),
    (dict(order=2, B_max=65, total_B=80), 2), (dict(total_B=1), 2), (dict(total_B=9), 2), (dict(order=3), 2), (dict(order=-1), 2),
    (dict(order=1), 2), (dict(order=1, node_size=65), 2), (dict(order=2, node_size=1), 2), (dict(node_size=4), 2),
    (dict(sm_scale=0.0), 2), (dict(sm_scale=NAN), 2), (dict(sm_scale=INF), 2), (dict(q_row=-8), 2), (dict(dtype=2), 4),
    (dict(q=None), 1), (dict(k_cache=None), 1), (dict(v_cache=None), 1), (dict(k_scale=None), 1), (dict(v_scale=None), 1),
    (dict(block_table=None), 1), (dict(k_new=None), 1), (dict(v_new=None), 1), (dict(tau=None), 1), (dict(lens=None), 1),
    (dict(cu_B=None), 1), (dict(out=None), 1), (dict(q=FAKE + 2), 8), (dict(out=FAKE + 8), 8), (dict(k_cache=FAKE + 4), 8),
    (dict(q_row=257), 8), (dict(k_row=132), 8), (dict(workspace=None), 5), (dict(workspace=FAKE + 8), 5),
    (dict(workspace_bytes=100), 5)])
def test_verify_refusals(lib, bad, code):
    d = verify_desc(**bad)
    assert lib.simsd_kvq_verify(ctypes.byref(d), None) == code
    assert (lib.simsd_kvq_verify_workspace_size(ctypes.byref(d)) == 0) == (code in (2, 4))
    assert lib.simsd_kvq_verify(None, None) == 1 and lib.simsd_kvq_verify_workspace_size(None) == 0


def test_verify_workspace_holds_partials_where_keys_are_split(lib):
    size = lambda **kw: lib.simsd_kvq_verify_workspace_size(ctypes.byref(verify_desc(**kw)))  # noqa: E731
    assert size(dtype=0) == 256                            # fp32, 64 keys: the status word alone
    assert size() % 256 == 0
    for dtype in (0, 1):
        short, long = (size(dtype=dtype, batch=1, total_B=4, max_pages_per_seq=m) for m in (4, 2048))
        # at least two splits of 8 rows x 4 heads: sums of 64 values, and (reference, sum)
        assert long - short >= 2 * 8 * 4 * (64 * 4 + 8)


def test_binding_refuses_what_it_would_misread():
    q = torch.zeros(4, 2, 64)
    ids = torch.zeros(4, dtype=torch.int32)
    spec = binding.rope_spec()
    with pytest.raises(ValueError):                        # a host tensor
        binding.rope(q, ids, spec, q)
    with pytest.raises(ValueError):                        # one of two second tensors
        binding.rope(q, ids, spec, q, q)
    with pytest.raises(ValueError):                        # a head's elements apart
        binding._heads_of(q.transpose(1, 2), q.dtype, 4, 2, "x")
    with pytest.raises(ValueError):                        # broadcast rows
        binding._row_stride(q[:1].expand(4, 2, 64), "k")
    with pytest.raises(ValueError):
        binding._row_stride(q.transpose(0, 1).contiguous().transpose(0, 1), "k")
    with pytest.raises(TypeError):
        binding._codes(k_cache=q)
    with pytest.raises(TypeError):
        binding._ints(torch.int32, lens=ids.long())
    with pytest.raises(ValueError):
        binding._ints(torch.int32, lens=torch.zeros(8, dtype=torch.int32)[::2])


@pytest.mark.parametrize("pack,desc", [("_PACK_ROPE", "RopeDesc"), ("_PACK_PAGE_MAP", "PageMapDesc"),
                                       ("_PACK_APPEND", "KvqAppendDesc"), ("_PACK_VERIFY", "KvqVerifyDesc")])
def test_packed_descriptors_are_the_structures(pack, desc):
    """Packing distinct values and reading them back through the structure gives the same values in the same fields."""
    fmt, cls = getattr(binding, pack), getattr(binding, desc)
    assert fmt.size == ctypes.sizeof(cls)
    spec = binding.rope_spec(base=7.0, rotary_dim=32, interleaved=True, scaling="yarn", factor=3.0, original_len=99)
    values = [bytes(spec) if f == "rope" else i + 1 for i, (f, _) in enumerate(cls._fields_)]
    d = cls.from_buffer_copy(fmt.pack(*values))
    for i, (f, _) in enumerate(cls._fields_):
        if f == "rope":
            assert bytes(d.rope) == bytes(spec) and d.rope.original_len == 99
        else:
            assert getattr(d, f) == i + 1, f
