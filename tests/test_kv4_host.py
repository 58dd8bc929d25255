"""Host side of the 4-bit-cache calls and of token_logprobs: descriptors, refusals,
workspace sizes, and the plain forms' own pins (no GPU needed, no kernel launched)."""
import ctypes
import os
import subprocess

import pytest
import torch

import kv4_ref as ref
from speculative_decoding_diffusion_gb300 import binding

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE = 1 << 20
DESCS = {"simsd_kv4_append_desc": binding.Kv4AppendDesc, "simsd_kv4_read_desc": binding.Kv4ReadDesc,
         "simsd_kv4_verify_desc": binding.Kv4VerifyDesc, "simsd_token_logprobs_desc": binding.TokenLogprobsDesc}


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


@pytest.mark.parametrize("pack,desc", [("_PACK_APPEND4", "Kv4AppendDesc"), ("_PACK_READ4", "Kv4ReadDesc"),
                                       ("_PACK_VERIFY4", "Kv4VerifyDesc"), ("_PACK_LOGPROBS", "TokenLogprobsDesc")])
def test_packed_descriptors_are_the_structures(pack, desc):
    fmt, cls = getattr(binding, pack), getattr(binding, desc)
    assert fmt.size == ctypes.sizeof(cls)
    spec = binding.rope_spec(base=7.0, rotary_dim=32, interleaved=True, scaling="yarn", factor=3.0, original_len=99)
    d = cls.from_buffer_copy(fmt.pack(*[bytes(spec) if f == "rope" else i + 1 for i, (f, _) in enumerate(cls._fields_)]))
    for i, (f, _) in enumerate(cls._fields_):
        assert bytes(d.rope) == bytes(spec) if f == "rope" else getattr(d, f) == i + 1, f


def test_exported(lib):
    for name in ("kv4_append", "kv4_read", "kv4_verify", "kv4_verify_workspace_size", "token_logprobs",
                 "token_logprobs_workspace_size"):
        assert hasattr(lib, "simsd_" + name)


def fill(d, **kw):
    for k, v in kw.items():
        setattr(d, k, v)
    return d


def append_desc(**kw):
    d = fill(binding.Kv4AppendDesc(), batch=2, num_kv_heads=2, head_dim=64, page_size=16, num_pages=8, max_pages_per_seq=4,
             total_n=5, dtype=1, rope=binding.rope_spec(base=1e4), k=FAKE, v=FAKE, start=FAKE, cu_n=FAKE, cache=FAKE,
             block_table=FAKE, workspace=FAKE, workspace_bytes=256)
    return fill(d, **kw)


def read_desc(**kw):
    d = fill(binding.Kv4ReadDesc(), batch=2, num_kv_heads=2, head_dim=64, page_size=16, num_pages=8, max_pages_per_seq=4,
             total_n=5, dtype=1, k=FAKE, v=FAKE, start=FAKE, cu_n=FAKE, cache=FAKE, block_table=FAKE, workspace=FAKE,
             workspace_bytes=256)
    return fill(d, **kw)


def verify_desc(**kw):
    d = fill(binding.Kv4VerifyDesc(), batch=2, num_q_heads=4, num_kv_heads=2, head_dim=64, page_size=16, num_pages=8,
             max_pages_per_seq=4, total_B=6, B_max=4, dtype=1, order=0, node_size=0, rope=binding.rope_spec(base=1e4),
             sm_scale=0.125, q=FAKE, cache=FAKE, block_table=FAKE, k_new=FAKE, v_new=FAKE, tau=FAKE, lens=FAKE, cu_B=FAKE,
             out=FAKE, workspace=FAKE, workspace_bytes=1 << 30)
    return fill(d, **kw)


def logprobs_desc(**kw):
    d = fill(binding.TokenLogprobsDesc(), rows=3, vocab=100, top_k=4, dtype=1, temperature=1.0, row_stride=0, logits=FAKE,
             tokens=FAKE, logprob=FAKE, rank=FAKE, entropy=FAKE, top_ids=FAKE, top_logprobs=FAKE, workspace=FAKE,
             workspace_bytes=1 << 20)
    return fill(d, **kw)


COMMON = [(dict(batch=0), 2), (dict(num_kv_heads=0), 2), (dict(head_dim=96), 2), (dict(page_size=32), 2),
          (dict(num_pages=0), 2), (dict(max_pages_per_seq=0), 2), (dict(block_table=None), 1), (dict(cache=None), 1),
          (dict(cache=FAKE + 8), 8), (dict(workspace=None), 5), (dict(workspace=FAKE + 16), 5), (dict(workspace_bytes=255), 5)]
ROWS = [(dict(total_n=-1), 2), (dict(total_n=(1 << 30) + 1), 2), (dict(k_row=-1), 2), (dict(num_kv_heads=1025), 2), (dict(batch=(1 << 20) + 1), 2),
        (dict(max_pages_per_seq=(1 << 26) + 1), 2), (dict(k=FAKE + 2), 8), (dict(v_row=130), 8), (dict(start=None), 1),
        (dict(cu_n=None), 1)]


@pytest.mark.parametrize("bad,code", COMMON + ROWS + [
    (dict(dtype=2), 4), (dict(k=None), 1), (dict(v=None), 1), (dict(rope=binding.rope_spec(base=0.5)), 2)])
def test_append_refusals(lib, bad, code):
    assert lib.simsd_kv4_append(ctypes.byref(append_desc(**bad)), None) == code


@pytest.mark.parametrize("bad,code", COMMON + ROWS + [
    (dict(dtype=3), 4), (dict(k=None, v=None), 1), (dict(k_row=64), 2), (dict(v_row=64), 2), (dict(dtype=2, k_row=136), 8)])
def test_read_refusals(lib, bad, code):
    assert lib.simsd_kv4_read(ctypes.byref(read_desc(**bad)), None) == code


@pytest.mark.parametrize("bad,code", COMMON + [
    (dict(dtype=2), 4), (dict(num_q_heads=3), 2), (dict(order=3), 2), (dict(node_size=2), 2), (dict(order=1, node_size=0), 2),
    (dict(B_max=33), 2), (dict(order=2, B_max=65), 2), (dict(total_B=1), 2), (dict(total_B=9), 2), (dict(sm_scale=0.0), 2),
    (dict(sm_scale=float("nan")), 2), (dict(q=None), 1), (dict(tau=None), 1), (dict(out=None), 1), (dict(k_new=FAKE + 2), 8),
    (dict(q_row=257), 8)])
def test_verify_refusals(lib, bad, code):
    assert lib.simsd_kv4_verify(ctypes.byref(verify_desc(**bad)), None) == code


@pytest.mark.parametrize("bad,code", [
    (dict(rows=-1), 2), (dict(rows=(1 << 20) + 1), 2), (dict(vocab=0), 2), (dict(vocab=(1 << 21) + 1), 2), (dict(top_k=-1), 2),
    (dict(top_k=33), 2), (dict(vocab=3), 2), (dict(dtype=2), 4), (dict(temperature=-1.0), 2),
    (dict(temperature=float("inf")), 2), (dict(temperature=2e30), 2), (dict(temperature=1e-31), 2), (dict(temperature=float("nan")), 2), (dict(row_stride=99), 2), (dict(logits=None), 1),
    (dict(tokens=None), 1), (dict(top_ids=None), 1), (dict(top_logprobs=None), 1), (dict(top_k=0), 1),
    (dict(logits=FAKE + 1), 8), (dict(dtype=0, logits=FAKE + 2), 8), (dict(workspace=None), 5),
    (dict(workspace_bytes=256 + 3 * 2 * 48 - 1), 5)])
def test_logprobs_refusals(lib, bad, code):
    assert lib.simsd_token_logprobs(ctypes.byref(logprobs_desc(**bad)), None) == code


def test_calls_without_rows(lib):
    assert lib.simsd_kv4_append(ctypes.byref(append_desc(total_n=0, k=None, v=None)), None) == 0
    assert lib.simsd_kv4_read(ctypes.byref(read_desc(total_n=0, k=None, v=None)), None) == 0
    assert lib.simsd_token_logprobs(ctypes.byref(logprobs_desc(rows=0, logits=None)), None) == 0
    for f in ("kv4_append", "kv4_read", "kv4_verify", "token_logprobs"):
        assert getattr(lib, "simsd_" + f)(None, None) == 1


@pytest.mark.parametrize("rows,vocab", [(0, 5), (1, 1), (3, 2048), (7, 2049), (1536, 151936), (1 << 20, 1 << 21)])
def test_logprobs_workspace_is_the_header_formula(lib, rows, vocab):
    want = (256 + rows * ((vocab + 2047) // 2048 + 1) * 48 + 255) // 256 * 256
    assert lib.simsd_token_logprobs_workspace_size(ctypes.byref(logprobs_desc(rows=rows, vocab=vocab, top_k=1))) == want


def test_verify_workspace_holds_partials_where_keys_are_split(lib):
    size = lambda **kw: lib.simsd_kv4_verify_workspace_size(ctypes.byref(verify_desc(**kw)))  # noqa: E731
    assert size(head_dim=96) == 0
    few = size(max_pages_per_seq=4096)                 # 4 units: cut; 1216 = 4 waves of two for each of 152 SMs: whole
    many = size(batch=608, total_B=1824, max_pages_per_seq=4096)
    assert few > 2 * 2 * 6 * 4 * 64 * 4 and many < 1 << 24


def test_binding_refuses_what_it_would_misread():
    q, ids, spec = torch.zeros(4, 2, 64), torch.zeros(5, dtype=torch.int32), binding.rope_spec()
    rec = torch.zeros(3, 2, 18 * 64, dtype=torch.uint8)
    for bad, error in ((rec.float(), TypeError), (rec.view(torch.int8), TypeError), (rec.transpose(0, 1), ValueError)):
        with pytest.raises(error):
            binding.kv4_append(q, q, ids[:1], ids[:2], bad, ids[:1].view(1, 1), ids, spec)
        with pytest.raises(error):
            binding.kv4_read(bad, ids[:1].view(1, 1), ids[:1], ids[:2], q, q, ids)
        with pytest.raises(error):
            binding.kv4_verify(q, bad, ids[:1].view(1, 1), q, q, None, ids[:1], ids[:2], q, ids, 4, 4, spec, 1.0, order=2)
    x, out = torch.zeros(4, 10), torch.zeros(4)
    for kw in (dict(logits=x.t()), dict(logits=x[:1].expand(4, 10)), dict(tokens=ids), dict(tokens=ids[:4].long()),
               dict(entropy=torch.zeros(3)), dict(rank=out), dict(top_ids=torch.zeros(4, 2, dtype=torch.int32)),
               dict(top_ids=torch.zeros(4, 2, dtype=torch.int32), top_logprobs=torch.zeros(4, 3))):
        args = dict(dict(logits=x, tokens=ids[:4], logprob=out, rank=None, entropy=None, top_ids=None, top_logprobs=None), **kw)
        with pytest.raises((ValueError, TypeError)):
            binding.token_logprobs_workspace_size(**args)
    assert binding.kv4_page_bytes(128) == 2304
    with pytest.raises(ValueError):
        binding.kv4_page_bytes(96)


def test_plain_form_of_the_format():
    """Against a search over every code and scale; pack and unpack are inverse."""
    g = torch.Generator().manual_seed(0)
    x = (torch.randn(40, 64, generator=g) * torch.exp2(torch.randint(-24, 18, (40, 1), generator=g).float())).double()
    byte = ref.scale_bytes(x)
    top = x.unflatten(-1, (-1, 16)).abs().amax(-1)
    best = (ref.SCALES[None, None] - (top / 6)[..., None]).abs().amin(-1)
    assert torch.equal((ref.scale_values(byte) - top / 6).abs(), best)
    code = ref.codes(x, byte)
    every = torch.cat([ref.CODES, -ref.CODES])[None, None, None] * ref.scale_values(byte)[..., None, None]
    best = (every - x.unflatten(-1, (-1, 16))[..., None]).abs().amin(-1).flatten(-2)
    assert torch.allclose((ref.values(code, byte) - x).abs(), best, rtol=1e-12, atol=0)
    for hd in (64, 128):
        rec = torch.randint(0, 256, (3, 2, 18 * hd), generator=g).to(torch.uint8)
        kc, kb, vc, vb = ref.unpack(rec)
        back = torch.zeros_like(rec)
        for p in range(3):
            for h in range(2):
                for i in range(16):
                    ref.put(back[p, h], 0, i, kc[p, h, i], kb[p, h, i])
                    ref.put(back[p, h], 1, i, vc[p, h, i], vb[p, h, i])
        assert torch.equal(back, rec)
