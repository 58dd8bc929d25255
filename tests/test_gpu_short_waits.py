"""Attention calls whose waits are allowed one to three polls: some give up with
products of the tensor cores and copies in flight.  A call sets the time-out bit or
is right, and so is the next call with the same workspace, however the one before
it ended."""
import math

import pytest
import torch

import kv4_ref
import speculative_decoding_diffusion_gb300 as pkg
import test_gpu_kv4 as kv4
import test_gpu_kvq as kvq

pytestmark = pytest.mark.gpu
TIMEOUT = 1


@pytest.mark.parametrize("B,lens", [(1, (900, 20)), (2, (3000, 0)), (4, (900, 700)), (8, (4000, 129)), (16, (20000, 40)), (32, (1000, 300))])
@pytest.mark.parametrize("hd", [128, 64])
def test_four_bit_cache(B, lens, hd):
    cache, table, cu, q, kn, vn, tau = kv4.case(B, lens, [B] * 2, "causal", "bf16", 4, 2, hd)
    args = (q.cuda(), cache.cuda(), table, kn.cuda(), vn.cuda(), None, lens, cu, B, dict(base=1e4), 1 / math.sqrt(hd), "causal")
    want, ws = kv4.verify(*args)
    assert pkg.read_status(ws) == 0
    exact, off = kv4_ref.verify(q, cache, table, kn, vn, tau, lens, cu, dict(base=1e4), 1 / math.sqrt(hd), "causal", 0, 2.0 ** -11)
    kv4.close(want, exact, off + 2.0 ** -32 * (max(lens) + 64) * 24, "bf16")
    for polls in (1, 2, 3) * 5:
        out, _ = kv4.verify(*args, wait_polls=polls, ws=ws)
        status = pkg.read_status(ws)
        assert status in (0, TIMEOUT) and (status or torch.equal(out, want))
        out, _ = kv4.verify(*args, ws=ws)
        assert pkg.read_status(ws) == 0 and torch.equal(out, want)


@pytest.mark.parametrize("B,lens", [(1, (900, 20)), (4, (900, 700)), (8, (4000, 129)), (16, (20000, 40)), (32, (1000, 300))])
@pytest.mark.parametrize("hd", [128, 64])
def test_eight_bit_cache(B, lens, hd):
    s = kvq.case(B, list(lens), [B] * 2, "causal", "bf16", 8, 2, hd)
    want, ws = kvq.launch(s)
    assert pkg.read_status(ws) == 0
    kvq.check(s, want)
    for polls in (1, 2, 3) * 5:
        out, _ = kvq.launch(s, ws=ws, polls=polls)
        status = pkg.read_status(ws)
        assert status in (0, TIMEOUT) and (status or torch.equal(out, want))
        out, _ = kvq.launch(s, ws=ws)
        assert pkg.read_status(ws) == 0 and torch.equal(out, want)


def test_paired_layout():
    from test_gpu_failure import DeviceWorkload, small_verify_workload
    dw = DeviceWorkload(small_verify_workload(seed=47), with_accept=False)
    args = (dw.q, dw.k_cache, dw.v_cache, dw.block_table, dw.k_new, dw.v_new, dw.tau, dw.lens, dw.cu_B, dw.out, dw.verify_ws,
            dw.total_B, dw.B_max, dw.rope_base, dw.sm_scale)
    pkg.verify_attn(*args)
    assert pkg.read_status(dw.verify_ws) == 0
    want = dw.out.clone()
    for polls in (1, 2, 3) * 5:
        pkg.verify_attn(*args, wait_polls=polls)
        status = pkg.read_status(dw.verify_ws)
        assert status in (0, TIMEOUT) and (status or torch.equal(dw.out, want))
        pkg.verify_attn(*args)
        assert pkg.read_status(dw.verify_ws) == 0 and torch.equal(dw.out, want)
